// Attention weight of cached keys (pe_kv_weigh): what attention over the 4-bit
// cache gives to each key, summed over a request's rows and the query heads of
// a key head, added to what the key had.
//
// The softmax's sums have to be known before a weight is, so the keys are read
// twice:
//  1. stats: per chunk of keys, the running maximum and sum of 2^score of every
//     row and head (a column);
//  2. join: the chunks' pairs of a column become its log2-sum;
//  3. weigh: scores again, and the sum over columns of 2^(score - log2-sum).
// Scores are K Q^T with the sixteen tokens of a record as the rows of an
// mma.sync m16n8k16 and eight columns as its columns: the sum over columns of pass
// 3 stays in registers, and a record is converted once for all columns.  Each key
// belongs to one warp: no atomics, the same result every time.
#include "pe_kv.cuh"

namespace pe {

struct WeighParams {
  int T, B, Hq, Hkv, G, block_size, bt_width, chunk, chunks;
  float scale2;  // scale * log2(e)
  long long num_blocks;
  const uint16_t* q;
  const uint8_t* cache;
  const int32_t* table;
  const int32_t* offsets;
  const int32_t* positions;
  const uint8_t* rejected;
  const float* mass;
  float* out;
  const int32_t* fresh;
  float2* parts;  // [chunks][T * Hq] maximum and sum
  float* lse;     // [T * Hq] log2 of the sum; +infinity: no weight
  uint32_t* err;
};

constexpr int kWeighThreads = 256;
constexpr int kWeighWarps = kWeighThreads / 32;
constexpr int kColBlock = 128;  // columns of one sweep over a chunk

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Keys that row t sees.
__device__ __forceinline__ int row_limit(const WeighParams& p, int t, bool report) {
  if (p.rejected && __ldg(p.rejected + t)) return 0;
  const int pos = __ldg(p.positions + t);
  const long long most = (long long)p.bt_width * p.block_size;
  if (pos < 0 || pos >= most) {
    if (report) atomicOr(p.err, PE_ERR_BLOCK_RANGE);
    return pos < 0 ? 0 : (int)most;
  }
  return pos + 1;
}
// Rows of request b (none where the offsets are out of order here).
__device__ __forceinline__ void request_rows(const WeighParams& p, int b, int& r0, int& r1) {
  if (p.offsets) {
    r0 = __ldg(p.offsets + b);
    r1 = __ldg(p.offsets + b + 1);
    if (r0 < 0 || r1 < r0 || r1 > p.T) r0 = r1 = 0;
  } else {
    r0 = b * (p.T / p.B);
    r1 = r0 + p.T / p.B;
  }
}

template <int D>
struct WeighShared {
  uint2 q[kColBlock / 8][D / 16][32];  // columns as B fragments, eight at a time
  float factor[kColBlock];  // scale * log2(e) and the power of two taken out of a column
  float lse[kColBlock];
  int limit[kColBlock];
  int most, least;          // of the columns' limits
  int reach;                // of all the request's rows
};

// One warp's lanes' part of a record's keys: rows g and g + 8, elements t D/4 .. (t+1) D/4
// (lane = 4 g + t), as loaded.
template <int D>
struct KeyWords {
  uint4 code[2];
  uint32_t scale[2];
  __device__ __forceinline__ void load(const uint8_t* rec, int lane) {
    using R = Record<D>;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint8_t* c = rec + R::kK + (g + 8 * i) * R::kRow + t * (D / 8);
      const uint8_t* s = rec + R::kKs + (g + 8 * i) * R::kScaleRow;
      if (D == 128) {
        code[i] = __ldg(reinterpret_cast<const uint4*>(c));
        scale[i] = __ldg(reinterpret_cast<const unsigned short*>(s) + t);
      } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(c));
        code[i] = make_uint4(v.x, v.y, 0u, 0u);
        scale[i] = __ldg(s + t);
      }
    }
  }
  // A fragments of the D/16 steps: step s takes the lane's elements 4 s .. 4 s + 3.
  __device__ __forceinline__ void convert(uint32_t (&a)[D / 16][4]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const uint32_t f = e4m3_f16x2((scale[i] >> (8 * (j / 2))) & 0xffu);
        uint32_t v[4];
        e2m1x8_f16(w[j], v);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          a[2 * j + h][i] = hmul2(v[2 * h], f);
          a[2 * j + h][2 + i] = hmul2(v[2 * h + 1], f);
        }
      }
    }
  }
};

// Columns c0.. of request rows [r0, r1), key head h, into shared memory.
template <int D>
__device__ __forceinline__ void load_columns(const WeighParams& p, WeighShared<D>& sh, int r0, int r1, int h, int c0, int n,
                                             bool weigh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) sh.most = 0, sh.least = INT32_MAX;
  __syncthreads();
  const int padded = (n + 7) & ~7;
  for (int c = warp; c < padded; c += kWeighWarps) {
    const bool live = c < n;
    const int row = r0 + (c0 + c) / p.G, head = h * p.G + (c0 + c) % p.G;
    uint2 w = make_uint2(0u, 0u);  // four elements, lane * 4 of D (D = 64: the upper half of the warp idles)
    if (live && 4 * lane < D)
      w = __ldg(reinterpret_cast<const uint2*>(p.q + ((long long)row * p.Hq + head) * D) + lane);
    float x[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
    float m = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
    // the power of two below the largest: 2^e <= m < 2^(e + 1)
    const int e = m > 0.f ? max((int)(__float_as_uint(m) >> 23) - 127, -100) : 0;
    const float down = __int_as_float((127 - min(e, 126)) << 23), up = __int_as_float((127 + min(e, 126)) << 23);
    uint32_t lo, hi;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(x[1] * down), "f"(x[0] * down));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(x[3] * down), "f"(x[2] * down));
    // element 4 lane = t D/4 + 4 s
    if (4 * lane < D) sh.q[c >> 3][lane % (D / 16)][4 * (c & 7) + lane / (D / 16)] = make_uint2(lo, hi);
    if (lane == 0) {
      const int limit = live ? row_limit(p, row, false) : 0;
      sh.factor[c] = p.scale2 * up;
      sh.limit[c] = limit;
      sh.lse[c] = live && weigh ? __ldcg(p.lse + (long long)row * p.Hq + head) : INFINITY;
      if (live) {
        atomicMax(&sh.most, limit);
        atomicMin(&sh.least, limit);
      }
    }
  }
  __syncthreads();
}

// The record of keys j0..j0+15 of request b and head h; NULL for a page outside the cache.
template <int D>
__device__ __forceinline__ const uint8_t* record_of(const WeighParams& p, int b, int h, int j0, long long& slot) {
  const int page = j0 / p.block_size, off = j0 - page * p.block_size;
  const long long block = __ldg(p.table + (long long)b * p.bt_width + page);
  slot = (block * p.Hkv + h) * p.block_size + off;
  if (block < 0 || block >= p.num_blocks) return nullptr;
  return p.cache + ((block * p.Hkv + h) * (p.block_size >> 4) + (off >> 4)) * (long long)Record<D>::kBytes;
}

template <int D, bool kWeigh>
__global__ void __launch_bounds__(kWeighThreads) weigh_kernel(const WeighParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  WeighShared<D>& sh = *reinterpret_cast<WeighShared<D>*>(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.y / p.Hkv, h = blockIdx.y - b * p.Hkv;
  const int chunk0 = blockIdx.x * p.chunk;
  int r0, r1;
  request_rows(p, b, r0, r1);
  if (r0 == r1) return;
  if (threadIdx.x == 0) sh.reach = 0;
  __syncthreads();
  int most = 0;
  for (int t = r0 + threadIdx.x; t < r1; t += kWeighThreads)
    most = max(most, row_limit(p, t, !kWeigh && h == 0 && blockIdx.x == 0));
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) atomicMax(&sh.reach, most);
  if (kWeigh) asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  const int reach = sh.reach;
  if (kWeigh && p.offsets && __ldcg(p.lse + (long long)p.T * p.Hq) != 0.f) return;  // offsets no partition
  if (chunk0 >= reach) return;
  const int chunk1 = min(reach, chunk0 + p.chunk);
  const int columns = (r1 - r0) * p.G;
  const int g = lane >> 2, t2 = 2 * (lane & 3);
  const int fresh = kWeigh && p.fresh ? __ldg(p.fresh + b) : INT32_MAX;

  for (int c0 = 0; c0 < columns; c0 += kColBlock) {
    const int n = min(kColBlock, columns - c0), tiles = (n + 7) >> 3;
    if (c0) __syncthreads();
    load_columns<D>(p, sh, r0, r1, h, c0, n, kWeigh);
    float m[kWeigh ? 1 : kColBlock / 8][2], l[kWeigh ? 1 : kColBlock / 8][2];
    if (!kWeigh) {
#pragma unroll
      for (int i = 0; i < (kWeigh ? 1 : kColBlock / 8); ++i) m[i][0] = m[i][1] = -INFINITY, l[i][0] = l[i][1] = 0.f;
    }
    long long slot, next_slot = 0;
    KeyWords<D> words;
    int j0 = chunk0 + 16 * warp;
    const uint8_t* rec = nullptr;
    if (j0 < chunk1) {
      rec = record_of<D>(p, b, h, j0, next_slot);
      if (rec) words.load(rec, lane);
    }
    for (; j0 < chunk1; j0 += 16 * kWeighWarps) {
      const uint8_t* cur = rec;
      slot = next_slot;
      uint32_t a[D / 16][4];
      if (cur) words.convert(a);
      if (j0 + 16 * kWeighWarps < chunk1) {  // the next record's loads ahead of this one's products
        rec = record_of<D>(p, b, h, j0 + 16 * kWeighWarps, next_slot);
        if (rec) words.load(rec, lane);
      }
      if (!cur) {
        if (!kWeigh && lane == 0) atomicOr(p.err, PE_ERR_BLOCK_RANGE);
        continue;
      }
      const bool edge = j0 + 16 > sh.least;
      float w0 = 0.f, w1 = 0.f;
#pragma unroll
      for (int i = 0; i < kColBlock / 8; ++i) {
        if (i < tiles) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint2 q = sh.q[i][s][lane];
            mma_f16(d, a[s], q.x, q.y);
          }
          const float2 f = *reinterpret_cast<const float2*>(&sh.factor[8 * i + t2]);
          d[0] *= f.x, d[1] *= f.y, d[2] *= f.x, d[3] *= f.y;
          if (edge) {
            const int2 lim = *reinterpret_cast<const int2*>(&sh.limit[8 * i + t2]);
            if (j0 + g >= lim.x) d[0] = -INFINITY;
            if (j0 + g >= lim.y) d[1] = -INFINITY;
            if (j0 + g + 8 >= lim.x) d[2] = -INFINITY;
            if (j0 + g + 8 >= lim.y) d[3] = -INFINITY;
          }
          if (kWeigh) {
            const float2 z = *reinterpret_cast<const float2*>(&sh.lse[8 * i + t2]);
            w0 += exp2_approx(d[0] - z.x) + exp2_approx(d[1] - z.y);
            w1 += exp2_approx(d[2] - z.x) + exp2_approx(d[3] - z.y);
          } else {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float& mm = m[kWeigh ? 0 : i][c];
              float& ll = l[kWeigh ? 0 : i][c];
              const float hi = fmaxf(d[c], d[c + 2]);
              if (hi > mm) {
                ll *= exp2_approx(mm - hi);
                mm = hi;
              }
              if (mm > -INFINITY) ll += exp2_approx(d[c] - mm) + exp2_approx(d[c + 2] - mm);
              else ll += d[c] + d[c + 2] == -INFINITY ? 0.f : d[c] + d[c + 2];  // a NaN stays one
            }
          }
        }
      }
      if (kWeigh) {
        w0 += __shfl_xor_sync(0xffffffffu, w0, 1);
        w1 += __shfl_xor_sync(0xffffffffu, w1, 1);
        w0 += __shfl_xor_sync(0xffffffffu, w0, 2);
        w1 += __shfl_xor_sync(0xffffffffu, w1, 2);
        if ((lane & 3) < 2) {
          const int r = g + 8 * (lane & 3), j = j0 + r;
          if (j < reach) {
            // columns past the first block add to what the blocks before them wrote
            float old = 0.f;
            if (c0) old = p.out[slot + r];
            else if (p.mass && j < fresh) old = p.mass[slot + r];
            p.out[slot + r] = old + ((lane & 3) ? w1 : w0);
          }
        }
      }
    }
    if (!kWeigh) {
      // a column's pair over the lanes of its quad column, then over the warps
      float2* join = reinterpret_cast<float2*>(smem + sizeof(WeighShared<D>));  // [warps][kColBlock]
#pragma unroll
      for (int i = 0; i < kColBlock / 8; ++i) {
        if (i < tiles) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mm = m[kWeigh ? 0 : i][c], ll = l[kWeigh ? 0 : i][c];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              const float m2 = __shfl_xor_sync(0xffffffffu, mm, o), l2 = __shfl_xor_sync(0xffffffffu, ll, o);
              const float hi = fmaxf(mm, m2);
              ll = ll * (mm == hi ? 1.f : exp2_approx(mm - hi)) + l2 * (m2 == hi ? 1.f : exp2_approx(m2 - hi));
              mm = hi;
            }
            if (g == 0) join[warp * kColBlock + 8 * i + t2 + c] = make_float2(mm, ll);
          }
        }
      }
      __syncthreads();
      for (int c = threadIdx.x; c < n; c += kWeighThreads) {
        float mm = -INFINITY, ll = 0.f;
        for (int w = 0; w < kWeighWarps; ++w) mm = fmaxf(mm, join[w * kColBlock + c].x);
        for (int w = 0; w < kWeighWarps; ++w) {
          const float2 v = join[w * kColBlock + c];
          ll += v.y * (v.x == mm ? 1.f : exp2_approx(v.x - mm));
        }
        const int row = r0 + (c0 + c) / p.G, head = h * p.G + (c0 + c) % p.G;
        p.parts[((long long)blockIdx.x * p.T + row) * p.Hq + head] = make_float2(mm, ll);
      }
    }
  }
}

// Column (row, head): the log2-sum over the chunks that its request reaches.
__global__ void __launch_bounds__(kWeighThreads) weigh_join_kernel(const WeighParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  bool ok = true;
  if (p.offsets) ok = offsets_valid(p.offsets, p.B, p.T, 0);
  const long long i = (long long)blockIdx.x * kWeighThreads + threadIdx.x;
  if (i == 0) {
    p.lse[(long long)p.T * p.Hq] = ok ? 0.f : 1.f;
    if (!ok) atomicOr(p.err, PE_ERR_OFFSETS);
  }
  if (i >= (long long)p.T * p.Hq) return;
  const int limit = row_limit(p, (int)(i / p.Hq), false);
  const int n = (limit + p.chunk - 1) / p.chunk;
  float m = -INFINITY, l = 0.f;
  for (int c = 0; c < n; ++c) {
    const float2 v = __ldcg(p.parts + (long long)c * p.T * p.Hq + i);
    const float hi = fmaxf(m, v.x);
    l = l * (m == hi ? 1.f : exp2_approx(m - hi)) + v.y * (v.x == hi ? 1.f : exp2_approx(v.x - hi));
    m = hi;
  }
  p.lse[i] = l == 0.f ? INFINITY : m + log2f(l);
}

}  // namespace pe

namespace {

// Keys of a chunk: as many as keep the GPU in work.
int weigh_chunk(int B, int Hkv, int64_t keys) {
  int chunk = 2048;
  while (chunk > 128 && (int64_t)B * Hkv * ((keys + chunk - 1) / chunk) < 4096) chunk /= 2;
  return chunk;
}

}  // namespace

extern "C" {

size_t pe_workspace_bytes_weigh(int32_t T, int32_t Hq, int32_t bt_width, int32_t block_size) {
  if (T < 0 || Hq < 1 || bt_width < 1 || block_size < 16 || (int64_t)bt_width * block_size > INT32_MAX) return 0;
  // (the smallest chunk)
  const size_t chunks = ((size_t)bt_width * block_size + 127) / 128, cols = (size_t)T * Hq;
  return (cols * 8 * chunks + (cols + 1) * 4 + 255) / 256 * 256;
}

int pe_kv_weigh(const pe_kv_weigh_args* a, void* stream) {
  if (!a) return PE_EINVAL;
  if (!pe_host::cache_sizes_ok(a->num_blocks, a->block_size, a->Hkv, a->D)) return PE_EINVAL;
  if (a->T < 0 || a->B < 1 || a->B > PE_MAX_ATTN_B || a->Hq < 1 || a->Hq % a->Hkv || a->Hq / a->Hkv > PE_MAX_ATTN_G)
    return PE_EINVAL;
  if (a->bt_width < 1 || (int64_t)a->bt_width * a->block_size > INT32_MAX) return PE_EINVAL;
  if ((int64_t)a->T * a->Hq > INT32_MAX / 2 || (int64_t)a->B * a->Hkv > 65535) return PE_EINVAL;
  if (!(a->scale > 0.f) || !(a->scale <= 3.0e38f)) return PE_EINVAL;
  if (!a->offsets && a->T % a->B) return PE_EINVAL;
  if (a->T == 0) return PE_OK;
  if (!a->q || !a->cache || !a->block_table || !a->positions || !a->out || !a->workspace || !a->err) return PE_EINVAL;
  if (!pe_host::aligned16(a->q) || !pe_host::aligned16(a->cache) || !pe_host::aligned16(a->workspace) ||
      !pe_host::aligned16(a->mass) || !pe_host::aligned16(a->out))
    return PE_EALIGN;
  pe::WeighParams p = {};
  p.T = a->T, p.B = a->B, p.Hq = a->Hq, p.Hkv = a->Hkv, p.G = a->Hq / a->Hkv;
  p.block_size = a->block_size, p.bt_width = a->bt_width;
  const int64_t keys = (int64_t)a->bt_width * a->block_size;
  p.chunk = weigh_chunk(a->B, a->Hkv, keys);
  p.chunks = (int)((keys + p.chunk - 1) / p.chunk);
  p.scale2 = (float)((double)a->scale * 1.4426950408889634);
  p.num_blocks = a->num_blocks;
  p.q = static_cast<const uint16_t*>(a->q);
  p.cache = static_cast<const uint8_t*>(a->cache);
  p.table = a->block_table, p.offsets = a->offsets, p.positions = a->positions, p.rejected = a->is_rejected;
  p.mass = a->mass, p.out = a->out, p.fresh = a->fresh;
  p.parts = static_cast<float2*>(a->workspace);
  p.lse = reinterpret_cast<float*>(p.parts + (size_t)p.chunks * p.T * p.Hq);
  p.err = a->err;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(p.chunks, p.B * p.Hkv);
  auto stats = a->D == 64 ? pe::weigh_kernel<64, false> : pe::weigh_kernel<128, false>;
  auto weigh = a->D == 64 ? pe::weigh_kernel<64, true> : pe::weigh_kernel<128, true>;
  const int fixed = a->D == 64 ? (int)sizeof(pe::WeighShared<64>) : (int)sizeof(pe::WeighShared<128>);
  const int join = fixed + (int)sizeof(float2) * pe::kWeighWarps * pe::kColBlock;
  static std::atomic<unsigned long long> done[4];
  if (!pe_host::allow_smem(stats, join, done[a->D == 64]) || !pe_host::allow_smem(weigh, fixed, done[2 + (a->D == 64)]))
    return PE_ECUDA;
  stats<<<grid, pe::kWeighThreads, join, st>>>(p);
  const unsigned cols = (unsigned)(((int64_t)p.T * p.Hq + pe::kWeighThreads - 1) / pe::kWeighThreads);
  pe::weigh_join_kernel<<<cols, pe::kWeighThreads, 0, st>>>(p);
  weigh<<<grid, pe::kWeighThreads, fixed, st>>>(p);
  return pe_host::launch_status();
}

}  // extern "C"
