// Rotated append to the 4-bit paged KV cache (pe_kv_append) and its read-back
// (pe_kv_read).
//
// Mathematics.  A pair (x0, x1) turns to (x0 c - x1 s, x1 c + x0 s).  A key is
// rounded to bf16 and its groups of 16 to e2m1 codes under an e4m3 scale.  Both
// roundings of keys are those of the exact value: a bf16 times an fp32 is a sum
// of two fp32 without error (product and fused remainder), the sum of two such
// products is brought to an fp32 rounded to odd, and that rounds to bf16 as the
// exact value would.  A rounding off by one in the last bit can move a key over a
// border of its code, to the next one; as it is, the cache holds what the key itself
// says, however a compiler contracts products.  Queries take plain fp32.
//
// Work.  A lane takes 32 elements of a head (two groups that hold both halves of
// its pairs), a warp 1024/D heads of keys and values or twice as many of queries,
// whose lanes use each table entry for two heads.  The warps go through all keys
// and values first, then through all queries: with both at once the two codes
// drove each other out of the instruction cache (200 us against 173 for the prompt rows
// below, three CTAs per SM).  Every element is read and written once.
//
// Measured (in a graph; D = 64, 64 + 16 heads, all dimensions rotated): 38 700 prompt
// rows 159 us, 4.9 TB/s of reads and writes, where the conversion's instructions and the
// loads wait for each other: the issue slots are 43 % busy, and loads in flight of 16
// warps an SM are what it waits for; two CTAs of 256 threads per SM (three: 168 us).
// 3584 decode rows of 32 + 8 heads of 128 15.5 us, 14 rows 3.6 us, a launch and one trip
// to memory.  The read-back: 23, 3.4 and 1.7 us of the same rows.
#include "pe_kv.cuh"

namespace pe {

struct AppendParams {
  int T, Hq, Hkv, block_size, half, max_pos, kv_chunks, q_chunks;
  long long slots_end;
  long long q_row, q_head, k_row, k_head, v_row, v_head;
  const uint16_t *q, *k, *v;
  const int32_t* positions;
  const long long* slots;
  const float* rope;
  uint8_t* cache;
  uint16_t *q_out, *k_out;
  uint32_t* err;
};

// x0 c - x1 s (or, with s negated and the roles swapped by the caller, the
// other half of the rotation) as the fp32 rounded to odd of the exact value.
__device__ __forceinline__ float diff_of_products_odd(float a, float c, float b, float s) {
  const float h1 = __fmul_rn(a, c), l1 = __fmaf_rn(a, c, -h1);
  const float h2 = __fmul_rn(b, s), l2 = __fmaf_rn(b, s, -h2);
  const float d = __fsub_rn(h1, h2);
  const float bb = __fsub_rn(d, h1);
  const float e = __fadd_rn(__fsub_rn(h1, __fsub_rn(d, bb)), -__fadd_rn(h2, bb));
  const float t = __fadd_rn(e, __fsub_rn(l1, l2));
  const float hi = __fadd_rn(d, t);
  const float tb = __fsub_rn(hi, d);
  const float lo = __fadd_rn(__fsub_rn(d, __fsub_rn(hi, tb)), __fsub_rn(t, tb));
  uint32_t u = __float_as_uint(hi);
  if (lo != 0.0f && !(u & 1u)) u += ((__float_as_uint(lo) ^ u) >> 31) ? 0xffffffffu : 1u;
  return lo == lo ? __uint_as_float(u) : d;  // an infinity has no remainder: all but d is a NaN
}

// 16 bf16 elements as codes (x, y) and scale (z) of one group.
__device__ __forceinline__ uint4 encode_group(uint4 a, uint4 b) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float x[16], m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
    m = fmaxf(m, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
  }
  // max / 6 lies on a border of e4m3 only when it is exact in fp32 (a border
  // has 5 significant bits, six times it 7, a bf16 has 8)
  const uint32_t scale = to_e4m3(fminf(__fdiv_rn(m, 6.0f), 448.0f));
  float s, unused;
  f16x2_to_f32(e4m3_f16x2(scale), s, unused);
  const float r = s > 0.0f ? __frcp_rn(s) : 0.0f;
  // x / s through the reciprocal, rounded to 16 significant bits: a quotient
  // that is not on a border of the code is 2^-9 away from it at least, one
  // that is on it has 4 bits, and comes out exact
#pragma unroll
  for (int i = 0; i < 16; ++i)
    x[i] = __uint_as_float((__float_as_uint(__fmul_rn(x[i], r)) + 0x80u) & 0xffffff00u);
  return make_uint4(to_e2m1x8(x), to_e2m1x8(x + 8), scale, 0);
}

// 32 elements of a head in two groups of 16.
struct Unit {
  uint32_t w[2][8];
  __device__ __forceinline__ void load(const uint16_t* head, int e0, int e1) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const uint4* v = reinterpret_cast<const uint4*>(head + (g ? e1 : e0));
      const uint4 a = v[0], b = v[1];
      w[g][0] = a.x, w[g][1] = a.y, w[g][2] = a.z, w[g][3] = a.w;
      w[g][4] = b.x, w[g][5] = b.y, w[g][6] = b.z, w[g][7] = b.w;
    }
  }
  __device__ __forceinline__ void store(uint16_t* head, int e0, int e1) const {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint4* v = reinterpret_cast<uint4*>(head + (g ? e1 : e0));
      v[0] = make_uint4(w[g][0], w[g][1], w[g][2], w[g][3]);
      v[1] = make_uint4(w[g][4], w[g][5], w[g][6], w[g][7]);
    }
  }
  // Turn pairs 4x .. 4x + 3 of the unit.
  template <bool kInterleaved, bool kExact>
  __device__ __forceinline__ void turn(int x, const float4& ca, const float4& sa) {
    const float c[4] = {ca.x, ca.y, ca.z, ca.w}, s[4] = {sa.x, sa.y, sa.z, sa.w};
    auto first = [](float a, float c, float b, float s) {
      return kExact ? diff_of_products_odd(a, c, b, s) : a * c - b * s;
    };
    if (kInterleaved) {
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        uint32_t& word = w[x / 2][4 * (x % 2) + y];
        const float x0 = bf16_lo(word), x1 = bf16_hi(word);
        word = pack_bf16(first(x0, c[y], x1, s[y]), first(x1, c[y], x0, -s[y]));
      }
    } else {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t &wa = w[0][2 * x + y], &wb = w[1][2 * x + y];
        const float a0 = bf16_lo(wa), a1 = bf16_hi(wa), b0 = bf16_lo(wb), b1 = bf16_hi(wb);
        const float c0 = c[2 * y], c1 = c[2 * y + 1], s0 = s[2 * y], s1 = s[2 * y + 1];
        wa = pack_bf16(first(a0, c0, b0, s0), first(a1, c1, b1, s1));
        wb = pack_bf16(first(b0, c0, a0, -s0), first(b1, c1, a1, -s1));
      }
    }
  }
};

template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 2) kv_append_kernel(const AppendParams p) {
  using R = Record<D>;
  constexpr int kUnits = D / 32, kHeads = 32 / kUnits;
  const int lane = threadIdx.x & 31;
  const int unit = lane % kUnits, head0 = lane / kUnits;
  const uint32_t nwarps = gridDim.x * (kThreads / 32);
  const uint32_t kv_items = (uint32_t)p.T * p.kv_chunks, items = kv_items + (uint32_t)p.T * p.q_chunks;
  // elements of the unit's two groups
  const bool turned = unit < p.half / 16;
  const int e0 = !turned ? 32 * unit : kInterleaved ? 32 * unit : 16 * unit;
  const int e1 = !turned || kInterleaved ? e0 + 16 : e0 + p.half;
  for (uint32_t it = (blockIdx.x * kThreads + threadIdx.x) >> 5; it < items; it += nwarps) {
    if (it < kv_items) {  // keys and values
      const int t = (int)(it / (uint32_t)p.kv_chunks), chunk = (int)(it - (uint32_t)t * p.kv_chunks);
      const int hh = chunk * kHeads + head0;
      const bool value = hh >= p.Hkv;
      const int h = value ? hh - p.Hkv : hh;
      const int pos = __ldg(p.positions + t);
      const long long slot = __ldg(p.slots + t);
      Unit u;
      if (hh < 2 * p.Hkv)
        u.load(value ? p.v + t * p.v_row + h * p.v_head : p.k + t * p.k_row + h * p.k_head, e0, e1);
      const bool pos_ok = pos >= 0 && pos < p.max_pos;
      const bool live = slot >= 0 && slot < p.slots_end;
      if (lane == 0 && chunk == 0) {
        if (!pos_ok) atomicOr(p.err, PE_ERR_POS_RANGE);
        if (!live && slot != -1) atomicOr(p.err, PE_ERR_BLOCK_RANGE);
      }
      if (hh >= 2 * p.Hkv) continue;
      if (!value) {
        if (turned && pos_ok) {
          const float4* cos_row =
              reinterpret_cast<const float4*>(p.rope + (long long)pos * 2 * p.half + 16 * unit);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            u.turn<kInterleaved, true>(x, __ldg(cos_row + x), __ldg(cos_row + p.half / 4 + x));
        }
        if (p.k_out) u.store(p.k_out + ((long long)t * p.Hkv + h) * D, e0, e1);
      }
      if (!live) continue;
      uint8_t* rec = p.cache + record_offset(slot, p.block_size, p.Hkv, h, R::kBytes);
      const int row = (int)(slot & 15);
      uint8_t* codes = rec + (value ? R::kV : R::kK) + row * R::kRow;
      uint8_t* scales = rec + (value ? R::kVs : R::kKs) + row * R::kScaleRow;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint4 c = encode_group(make_uint4(u.w[g][0], u.w[g][1], u.w[g][2], u.w[g][3]),
                                     make_uint4(u.w[g][4], u.w[g][5], u.w[g][6], u.w[g][7]));
        const int e = g ? e1 : e0;
        *reinterpret_cast<uint2*>(codes + e / 2) = make_uint2(c.x, c.y);
        scales[e / 16] = (uint8_t)c.z;
      }
    } else {  // queries, two heads per lane
      const uint32_t rest = it - kv_items;
      const int t = (int)(rest / (uint32_t)p.q_chunks), chunk = (int)(rest - (uint32_t)t * p.q_chunks);
      const int h = chunk * 2 * kHeads + head0;
      const int pos = __ldg(p.positions + t);
      Unit u[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (h + i * kHeads < p.Hq) u[i].load(p.q + t * p.q_row + (h + i * kHeads) * p.q_head, e0, e1);
      if (turned && pos >= 0 && pos < p.max_pos) {
        const float4* cos_row =
            reinterpret_cast<const float4*>(p.rope + (long long)pos * 2 * p.half + 16 * unit);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float4 c = __ldg(cos_row + x), s = __ldg(cos_row + p.half / 4 + x);
#pragma unroll
          for (int i = 0; i < 2; ++i) u[i].turn<kInterleaved, false>(x, c, s);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (h + i * kHeads < p.Hq) u[i].store(p.q_out + ((long long)t * p.Hq + h + i * kHeads) * D, e0, e1);
    }
  }
}

// One thread per group of 16 elements of one row and head, keys and values.
template <int D>
__global__ void __launch_bounds__(kThreads)
    kv_read_kernel(const uint8_t* cache, long long slots_end, int block_size, int Hkv,
                   const long long* slots, int n, uint16_t* k_out, uint16_t* v_out, uint32_t* err) {
  using R = Record<D>;
  const uint32_t total = (uint32_t)n * Hkv * (D / 8);  // the host keeps it below 2^32
  for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < total; i += gridDim.x * kThreads) {
    const int g = (int)(i % (D / 16));
    const uint32_t rest = i / (D / 16);
    const int kind = (int)(rest & 1);
    const uint32_t row = rest >> 1;  // t * Hkv + h
    const int t = (int)(row / (uint32_t)Hkv), h = (int)(row - (uint32_t)t * Hkv);
    uint16_t* out = kind ? v_out : k_out;
    const long long slot = __ldg(slots + t);
    const bool live = slot >= 0 && slot < slots_end;
    if (!live && slot != -1 && g == 0 && kind == 0 && h == 0) atomicOr(err, PE_ERR_BLOCK_RANGE);
    if (!out) continue;
    uint32_t w[8] = {};
    if (live) {
      const uint8_t* rec = cache + record_offset(slot, block_size, Hkv, h, R::kBytes);
      const int r = (int)(slot & 15);
      const uint2 codes =
          *reinterpret_cast<const uint2*>(rec + (kind ? R::kV : R::kK) + r * R::kRow + 8 * g);
      const uint32_t s = e4m3_f16x2(rec[(kind ? R::kVs : R::kKs) + r * R::kScaleRow + g]);
      uint32_t a[4], b[4];
      e2m1x8_f16(codes.x, a);
      e2m1x8_f16(codes.y, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float lo, hi;  // at most 6 significant bits: exact in f16 and in bf16
        f16x2_to_f32(hmul2(j < 4 ? a[j & 3] : b[j & 3], s), lo, hi);
        w[j] = pack_bf16(lo, hi);
      }
    }
    uint4* v = reinterpret_cast<uint4*>(out + (long long)row * D + 16 * g);
    v[0] = make_uint4(w[0], w[1], w[2], w[3]);
    v[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

}  // namespace pe

namespace {

bool strides_ok(int64_t row, int64_t head) { return row >= 0 && head >= 0 && row % 8 == 0 && head % 8 == 0; }

}  // namespace

extern "C" int pe_kv_append(const pe_kv_append_args* a, void* stream) {
  if (!a) return PE_EINVAL;
  if (!pe_host::cache_sizes_ok(a->num_blocks, a->block_size, a->Hkv, a->D)) return PE_EINVAL;
  if (a->T < 0 || a->Hq < 1 || a->Hq % a->Hkv) return PE_EINVAL;
  if (a->T > INT32_MAX / 16 / ((int64_t)a->Hq + 2 * (int64_t)a->Hkv)) return PE_EINVAL;
  if (a->rot_dim < 32 || a->rot_dim > a->D || a->rot_dim % 32 || a->max_pos < 1) return PE_EINVAL;
  if (a->T == 0) return PE_OK;
  if (!a->q || !a->k || !a->v || !a->positions || !a->slots || !a->rope || !a->cache || !a->q_out ||
      !a->err)
    return PE_EINVAL;
  const void* ptrs[] = {a->q, a->k, a->v, a->rope, a->cache, a->q_out, a->k_out};
  for (const void* x : ptrs)
    if (!pe_host::aligned16(x)) return PE_EALIGN;
  if (!strides_ok(a->q_row, a->q_head) || !strides_ok(a->k_row, a->k_head) ||
      !strides_ok(a->v_row, a->v_head))
    return PE_EALIGN;
  pe_host::DeviceInfo dev;
  if (pe_host::device_info(&dev) != PE_OK) return PE_ECUDA;
  pe::AppendParams p;
  p.T = a->T, p.Hq = a->Hq, p.Hkv = a->Hkv, p.block_size = a->block_size;
  p.half = a->rot_dim / 2, p.max_pos = a->max_pos;
  p.slots_end = a->num_blocks * a->block_size;
  p.q_row = a->q_row, p.q_head = a->q_head, p.k_row = a->k_row, p.k_head = a->k_head;
  p.v_row = a->v_row, p.v_head = a->v_head;
  p.q = static_cast<const uint16_t*>(a->q);
  p.k = static_cast<const uint16_t*>(a->k);
  p.v = static_cast<const uint16_t*>(a->v);
  p.positions = a->positions;
  p.slots = reinterpret_cast<const long long*>(a->slots);
  p.rope = a->rope;
  p.cache = static_cast<uint8_t*>(a->cache);
  p.q_out = static_cast<uint16_t*>(a->q_out);
  p.k_out = static_cast<uint16_t*>(a->k_out);
  p.err = a->err;
  const int per_warp = 1024 / a->D;
  p.kv_chunks = (2 * a->Hkv + per_warp - 1) / per_warp;
  p.q_chunks = (a->Hq + 2 * per_warp - 1) / (2 * per_warp);
  const long long warps = (long long)a->T * (p.kv_chunks + p.q_chunks);
  const long long want = (warps + pe::kWarps - 1) / pe::kWarps;
  const long long most = (long long)dev.sm_count * 8;
  const int grid = (int)(want < most ? want : most);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto kernel = a->D == 64 ? (a->interleaved ? pe::kv_append_kernel<64, true> : pe::kv_append_kernel<64, false>)
                           : (a->interleaved ? pe::kv_append_kernel<128, true> : pe::kv_append_kernel<128, false>);
  kernel<<<grid, pe::kThreads, 0, s>>>(p);
  return pe_host::launch_status();
}

extern "C" int pe_kv_read(const void* cache, int64_t num_blocks, int32_t block_size, int32_t Hkv,
                          int32_t D, const int64_t* slots, int32_t n, void* k_out, void* v_out,
                          uint32_t* err, void* stream) {
  if (!pe_host::cache_sizes_ok(num_blocks, block_size, Hkv, D)) return PE_EINVAL;
  if (n < 0 || (int64_t)n * Hkv > INT32_MAX / 32) return PE_EINVAL;
  if (n == 0) return PE_OK;
  if (!cache || !slots || !err) return PE_EINVAL;
  if (!pe_host::aligned16(cache) || !pe_host::aligned16(k_out) || !pe_host::aligned16(v_out))
    return PE_EALIGN;
  pe_host::DeviceInfo dev;
  if (pe_host::device_info(&dev) != PE_OK) return PE_ECUDA;
  const long long want = ((long long)n * Hkv * 2 * (D / 16) + pe::kThreads - 1) / pe::kThreads;
  const long long most = (long long)dev.sm_count * 8;
  const int grid = (int)(want < most ? want : most);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const uint8_t* c = static_cast<const uint8_t*>(cache);
  const long long* sl = reinterpret_cast<const long long*>(slots);
  uint16_t *ko = static_cast<uint16_t*>(k_out), *vo = static_cast<uint16_t*>(v_out);
  const long long slots_end = num_blocks * (int64_t)block_size;
  if (D == 64)
    pe::kv_read_kernel<64><<<grid, pe::kThreads, 0, s>>>(c, slots_end, block_size, Hkv, sl, n, ko, vo, err);
  else
    pe::kv_read_kernel<128><<<grid, pe::kThreads, 0, s>>>(c, slots_end, block_size, Hkv, sl, n, ko, vo, err);
  return pe_host::launch_status();
}
