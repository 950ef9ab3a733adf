// Rotated append to the 4-bit paged KV cache (pe_kv_append) and its read-back
// (pe_kv_read).
//
// Mathematics.  A pair (x0, x1) turns to (x0 c - x1 s, x1 c + x0 s).  A key is
// rounded to bf16 and its groups of 16 to e2m1 codes under an e4m3 scale.  Both
// roundings of keys are those of the exact value: a bf16 times an fp32 is a sum
// of two fp32 without error (product and fused remainder), the sum of two such
// products is brought to an fp32 rounded to odd, and that rounds to bf16 as the
// exact value would.  So a key next to a border of its code falls on the right
// side, whatever order a checker adds in.  Queries take plain fp32.
//
// Work.  A warp takes one row; its lanes are D/32 units of 32 elements times
// 1024/D heads, so a lane keeps the 32 table entries of its unit for every
// head that it visits.  Queries, keys and values are one list of heads.  Bound
// by memory: every element is read and written once.
#include "pe_kv.cuh"

namespace pe {

struct AppendParams {
  int T, Hq, Hkv, block_size, half, interleaved, max_pos, chunks;
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
  return lo == lo ? __uint_as_float(u) : hi;  // an infinity or NaN leaves no remainder
}

// 16 bf16 elements (8 words) as codes and scale of one group.
__device__ __forceinline__ void encode_group(const uint32_t (&w)[8], uint2& codes, uint32_t& scale) {
  float x[16], m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
    m = fmaxf(m, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
  }
  // max / 6 lies on a border of e4m3 only when it is exact in fp32 (a border
  // has 5 significant bits, six times it 7, a bf16 has 8)
  scale = to_e4m3(fminf(__fdiv_rn(m, 6.0f), 448.0f));
  float s, unused;
  f16x2_to_f32(e4m3_f16x2(scale), s, unused);
  const float r = s > 0.0f ? __frcp_rn(s) : 0.0f;
  // x / s through the reciprocal, rounded to 16 significant bits: a quotient
  // that is not on a border of the code is 2^-9 away from it at least, one
  // that is on it has 4 bits, and comes out exact
#pragma unroll
  for (int i = 0; i < 16; ++i)
    x[i] = __uint_as_float((__float_as_uint(__fmul_rn(x[i], r)) + 0x80u) & 0xffffff00u);
  codes.x = to_e2m1x8(x);
  codes.y = to_e2m1x8(x + 8);
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendParams p) {
  using R = Record<D>;
  constexpr int kUnits = D / 32, kHeads = 32 / kUnits;
  const int lane = threadIdx.x & 31;
  const int unit = lane % kUnits, head0 = lane / kUnits;
  const long long nwarps = ((long long)gridDim.x * kThreads) >> 5;
  const int heads = p.Hq + 2 * p.Hkv;
  const int per_chunk = (heads + p.chunks - 1) / p.chunks;
  const int rot_units = p.half / 16;
  // elements of the unit's two groups
  const bool turned = unit < rot_units;
  const int e0 = !turned ? 32 * unit : p.interleaved ? 32 * unit : 16 * unit;
  const int e1 = !turned || p.interleaved ? e0 + 16 : e0 + p.half;
  for (long long it = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
       it < (long long)p.T * p.chunks; it += nwarps) {
    const int t = (int)(it / p.chunks), chunk = (int)(it - (long long)t * p.chunks);
    const int pos = __ldg(p.positions + t);
    const long long slot = __ldg(p.slots + t);
    const bool pos_ok = pos >= 0 && pos < p.max_pos;
    const bool live = slot >= 0 && slot < p.slots_end;
    if (lane == 0 && chunk == 0) {
      if (!pos_ok) atomicOr(p.err, PE_ERR_POS_RANGE);
      if (!live && slot != -1) atomicOr(p.err, PE_ERR_BLOCK_RANGE);
    }
    const bool turn = turned && pos_ok;
    float c[16], s[16];
    if (turn) {
      const float4* row = reinterpret_cast<const float4*>(p.rope + (long long)pos * 2 * p.half +
                                                          16 * unit);
      const float4* sin_row = row + p.half / 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 a = __ldg(row + i), b = __ldg(sin_row + i);
        c[4 * i] = a.x, c[4 * i + 1] = a.y, c[4 * i + 2] = a.z, c[4 * i + 3] = a.w;
        s[4 * i] = b.x, s[4 * i + 1] = b.y, s[4 * i + 2] = b.z, s[4 * i + 3] = b.w;
      }
    }
    const int end = min(heads, (chunk + 1) * per_chunk);
    for (int hh = chunk * per_chunk + head0; hh < end; hh += kHeads) {
      const int kind = hh < p.Hq ? 0 : hh < p.Hq + p.Hkv ? 1 : 2;
      const int h = kind == 0 ? hh : hh - p.Hq - (kind == 2 ? p.Hkv : 0);
      const uint16_t* src = kind == 0   ? p.q + t * p.q_row + h * p.q_head
                            : kind == 1 ? p.k + t * p.k_row + h * p.k_head
                                        : p.v + t * p.v_row + h * p.v_head;
      uint32_t w[2][8];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint4* v = reinterpret_cast<const uint4*>(src + (g ? e1 : e0));
        const uint4 a = v[0], b = v[1];
        w[g][0] = a.x, w[g][1] = a.y, w[g][2] = a.z, w[g][3] = a.w;
        w[g][4] = b.x, w[g][5] = b.y, w[g][6] = b.z, w[g][7] = b.w;
      }
      if (kind < 2) {
        if (turn) {
          if (p.interleaved) {
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float x0 = bf16_lo(w[g][i]), x1 = bf16_hi(w[g][i]);
                const float ci = c[8 * g + i], si = s[8 * g + i];
                w[g][i] = kind == 0 ? pack_bf16(x0 * ci - x1 * si, x1 * ci + x0 * si)
                                    : pack_bf16(diff_of_products_odd(x0, ci, x1, si),
                                                diff_of_products_odd(x1, ci, x0, -si));
              }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float a0 = bf16_lo(w[0][i]), a1 = bf16_hi(w[0][i]);
              const float b0 = bf16_lo(w[1][i]), b1 = bf16_hi(w[1][i]);
              const float c0 = c[2 * i], c1 = c[2 * i + 1], s0 = s[2 * i], s1 = s[2 * i + 1];
              if (kind == 0) {
                w[0][i] = pack_bf16(a0 * c0 - b0 * s0, a1 * c1 - b1 * s1);
                w[1][i] = pack_bf16(b0 * c0 + a0 * s0, b1 * c1 + a1 * s1);
              } else {
                w[0][i] = pack_bf16(diff_of_products_odd(a0, c0, b0, s0),
                                    diff_of_products_odd(a1, c1, b1, s1));
                w[1][i] = pack_bf16(diff_of_products_odd(b0, c0, a0, -s0),
                                    diff_of_products_odd(b1, c1, a1, -s1));
              }
            }
          }
        }
        uint16_t* out = kind == 0 ? p.q_out + ((long long)t * p.Hq + h) * D
                        : p.k_out ? p.k_out + ((long long)t * p.Hkv + h) * D
                                  : nullptr;
        if (out) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint4* v = reinterpret_cast<uint4*>(out + (g ? e1 : e0));
            v[0] = make_uint4(w[g][0], w[g][1], w[g][2], w[g][3]);
            v[1] = make_uint4(w[g][4], w[g][5], w[g][6], w[g][7]);
          }
        }
      }
      if (kind > 0 && live) {
        uint8_t* rec = p.cache + record_offset(slot, p.block_size, p.Hkv, h, R::kBytes);
        const int row = (int)(slot & 15);
        uint8_t* codes = rec + (kind == 1 ? R::kK : R::kV) + row * R::kRow;
        uint8_t* scales = rec + (kind == 1 ? R::kKs : R::kVs) + row * R::kScaleRow;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint2 cd;
          uint32_t sc;
          encode_group(w[g], cd, sc);
          const int e = g ? e1 : e0;
          *reinterpret_cast<uint2*>(codes + e / 2) = cd;
          scales[e / 16] = (uint8_t)sc;
        }
      }
    }
  }
}

// One thread per group of 16 elements of one row and head, keys and values.
template <int D>
__global__ void __launch_bounds__(kThreads)
    kv_read_kernel(const uint8_t* cache, long long slots_end, int block_size, int Hkv,
                   const long long* slots, int n, uint16_t* k_out, uint16_t* v_out, uint32_t* err) {
  using R = Record<D>;
  const long long total = (long long)n * Hkv * 2 * (D / 16);
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < total;
       i += (long long)gridDim.x * kThreads) {
    const int g = (int)(i % (D / 16));
    const long long rest = i / (D / 16);
    const int kind = (int)(rest & 1);
    const long long row = rest >> 1;  // t * Hkv + h
    const int t = (int)(row / Hkv), h = (int)(row - (long long)t * Hkv);
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
    uint4* v = reinterpret_cast<uint4*>(out + row * D + 16 * g);
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
  if (a->T < 0 || a->Hq < 1 || a->Hkv < 1 || a->Hq % a->Hkv || (a->D != 64 && a->D != 128))
    return PE_EINVAL;
  if (a->block_size < 16 || a->block_size % 16 || a->num_blocks < 1 ||
      a->num_blocks > (INT64_MAX >> 8) / ((int64_t)a->Hkv * a->block_size * a->D))
    return PE_EINVAL;
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
  p.half = a->rot_dim / 2, p.interleaved = a->interleaved != 0, p.max_pos = a->max_pos;
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
  const int heads = a->Hq + 2 * a->Hkv, per_warp = 1024 / a->D;
  p.chunks = (heads + per_warp - 1) / per_warp;
  const long long warps = (long long)a->T * p.chunks;
  const long long want = (warps + pe::kWarps - 1) / pe::kWarps;
  const long long most = (long long)dev.sm_count * 8;
  const int grid = (int)(want < most ? want : most);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->D == 64)
    pe::kv_append_kernel<64><<<grid, pe::kThreads, 0, s>>>(p);
  else
    pe::kv_append_kernel<128><<<grid, pe::kThreads, 0, s>>>(p);
  return pe_host::launch_status();
}

extern "C" int pe_kv_read(const void* cache, int64_t num_blocks, int32_t block_size, int32_t Hkv,
                          int32_t D, const int64_t* slots, int32_t n, void* k_out, void* v_out,
                          uint32_t* err, void* stream) {
  if (n < 0 || Hkv < 1 || (D != 64 && D != 128) || block_size < 16 || block_size % 16 ||
      num_blocks < 1 || num_blocks > (INT64_MAX >> 8) / ((int64_t)Hkv * block_size * D))
    return PE_EINVAL;
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
