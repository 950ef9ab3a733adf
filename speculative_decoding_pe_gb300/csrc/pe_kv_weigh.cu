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
//
// One token, 256 requests of up to 65,535 keys, 4 heads of 128: 1.21 ms, 66 % of two reads at the copy
// rate; issue slots (75 % busy) bound it, of which converting codes takes the most.  64 drafts of 14 rows,
// up to 32,767 keys, 8 heads of 64: 0.77 ms, 7 % of the bytes' floor; products and exponentials wait
// for each other at 16 warps an SM (mma.sync 36 % busy, ex2 19 %).
#include <type_traits>

#include "pe_cluster.cuh"
#include "pe_kv.cuh"
#include "pe_tma.cuh"

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
constexpr int kLiveRows = 64;   // (a draft batch's rejected rows are no columns)
constexpr int kStages = 4;      // records of a warp on their way

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

// Two products, two sums in one instruction each.  The products as x y + zero with a zero that
// the compiler does not know: a packed product with a sum directly after it was compiled
// into one fused operation, although both say .rn.
__device__ __forceinline__ void mul2(float& d0, float& d1, float2 f, float zero) {
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tmov.b64 c, {%4, %4};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(d0), "+f"(d1)
      : "f"(f.x), "f"(f.y), "f"(zero));
}
__device__ __forceinline__ float2 add2(float d0, float d1, float2 z) {
  float2 r;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 a, a, b;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(d0), "f"(d1), "f"(z.x), "f"(z.y));
  return r;
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

// kTiles: tiles of eight columns that one look takes.
template <int D, int kTiles>
struct WeighShared {
  static constexpr int kCols = 8 * kTiles;
  static constexpr int kCodes = 16 * Record<D>::kRow, kScales = 16 * Record<D>::kScaleRow;
  uint8_t ring[kWeighWarps][kStages][kCodes + kScales];  // the keys of records
  uint4 q[kTiles][D / 32][32];  // columns as B fragments, eight at a time, two steps in a word
  uint64_t bars[kWeighWarps][kStages];
  float factor[kCols];  // scale * log2(e) and the power of two taken out of a column
  float lse[kCols];     // minus the log2-sum of a column; -infinity: no weight
  int limit[kCols];
  float2 sums[kCols];   // this CTA's maximum and sum of a column
  float2 join[kWeighWarps][kCols];
  int rows[kLiveRows];  // the request's rows that see any key, where it has so few in all
  int live;
  int least;            // of the columns' limits
  int reach;            // of all the request's rows
};

// One warp's lanes' part of a record's keys: rows g and g + 8, elements t D/4 .. (t+1) D/4
// (lane = 4 g + t), as loaded.
template <int D>
struct KeyWords {
  uint4 code[2];
  uint32_t scale[2];
  __device__ __forceinline__ void load(const uint8_t* keys, int lane) {  // codes, then scales
    using R = Record<D>;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint8_t* c = keys + (g + 8 * i) * R::kRow + t * (D / 8);
      const uint8_t* s = keys + 16 * R::kRow + (g + 8 * i) * R::kScaleRow;
      if (D == 128) {
        code[i] = *reinterpret_cast<const uint4*>(c);
        scale[i] = reinterpret_cast<const unsigned short*>(s)[t];
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(c);
        code[i] = make_uint4(v.x, v.y, 0u, 0u);
        scale[i] = s[t];
      }
    }
  }
  // A fragments of the D/16 steps: step s takes the lane's elements 4 s .. 4 s + 3.
  __device__ __forceinline__ void convert(uint32_t (&a)[D / 16][4]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
      const uint32_t both = e4m3x2_f16x2(scale[i]);  // the scales of the lane's two groups (D = 64: one)
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const uint32_t f = __byte_perm(both, 0, j < 2 ? 0x1010 : 0x3232);
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

// Columns c0.. of the request's rows from r0 on, key head h, into shared memory.
template <int D, int kTiles>
__device__ __forceinline__ void load_columns(const WeighParams& p, WeighShared<D, kTiles>& sh, int r0, bool listed, int h, int c0, int n) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();  // the last sweep's readers
  if (threadIdx.x == 0) sh.least = INT32_MAX;
  __syncthreads();
  const int padded = kTiles == 1 ? 8 : (n + 15) & ~15;  // (whole pairs of tiles)
  for (int c = warp; c < padded; c += kWeighWarps) {
    const bool live = c < n;
    const int of = (c0 + c) / p.G, head = h * p.G + (c0 + c) % p.G;
    const int row = !live ? 0 : listed ? sh.rows[of] : r0 + of;
    const int limit = live ? row_limit(p, row, false) : 0;
    // four elements, lane * 4 of D (D = 64: the upper half of the warp idles); a row that sees nothing
    // is a column of zeros: what its query holds, a NaN too, reaches no key
    uint2 w = make_uint2(0u, 0u);
    if (limit && 4 * lane < D)
      w = __ldg(reinterpret_cast<const uint2*>(p.q + ((long long)row * p.Hq + head) * D) + lane);
    float x[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
    float m = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
    // Not finite: NaN as a whole.  (An infinity alone may give -infinity with every key, which
    // would count as a row that sees nothing.)
    if (m == INFINITY) x[0] = x[1] = x[2] = x[3] = NAN;
    // the power of two below the largest: 2^e <= m < 2^(e + 1)
    const int e = m > 0.f ? max((int)(__float_as_uint(m) >> 23) - 127, -100) : 0;
    const float down = __int_as_float((127 - min(e, 126)) << 23), up = __int_as_float((127 + min(e, 126)) << 23);
    uint32_t lo, hi;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(x[1] * down), "f"(x[0] * down));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(x[3] * down), "f"(x[2] * down));
    // element 4 lane = t D/4 + 4 s
    const int s = lane % (D / 16);
    if (4 * lane < D)
      reinterpret_cast<uint2*>(&sh.q[c >> 3][s >> 1][4 * (c & 7) + lane / (D / 16)])[s & 1] = make_uint2(lo, hi);
    if (lane == 0) {
      sh.factor[c] = fmaxf(p.scale2 * up, 1.2e-38f);  // (above 0: an infinity times it is one)
      sh.limit[c] = limit;
      sh.lse[c] = -INFINITY;
      if (limit) atomicMin(&sh.least, limit);  // (a column that sees nothing gets no weight by its lse)
    }
  }
  __syncthreads();
}

constexpr float kLowest = -3.4e38f;  // below every score (finite: nothing less it is no NaN)

// Sum of 2^(score - m) of two columns of each tile, over a lane's rows.  m is the larger
// score of the lane's first two rows, which any later one may pass: the sum is a float, and only
// where it grew by more than 2^100 the look is repeated with a running maximum (which takes half
// as many instructions again).
template <int kTiles>
struct Stats {
  float m[kTiles][2], l[kTiles][2];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kTiles; ++i) m[i][0] = m[i][1] = kLowest, l[i][0] = l[i][1] = 0.f;
  }
};

// One look at the records [rec0, rec1) of request b, key head h, by this CTA's warps.  A
// record's sixteen tokens against all columns: kWeigh: the sum over columns of
// 2^(score - lse) goes to out; else the columns' statistics.
template <int D, int kTiles, bool kWeigh>
__device__ __forceinline__ void sweep(const WeighParams& p, WeighShared<D, kTiles>& sh, int b, int h, int rec0, int rec1, int reach,
                                      int tiles, bool more, bool track, uint32_t& turn, Stats<kTiles>& st) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t2 = 2 * (lane & 3);
  const int fresh = kWeigh && p.fresh ? __ldg(p.fresh + b) : INT32_MAX;
  const int page_recs = p.block_size >> 4;
  const float zero = __int_as_float((int)(0x80000000u | ((uint32_t)p.T >> 31)));  // -0: T is not negative
  const int32_t* table = p.table + (long long)b * p.bt_width;
  uint4 q1[D / 32];  // one tile's columns stay in registers
  if (kTiles == 1) {
#pragma unroll
    for (int s = 0; s < D / 32; ++s) q1[s] = sh.q[0][s][lane];
  }
  for (int r0 = rec0 + warp; r0 < rec1; r0 += 32 * kWeighWarps) {
    // where the warp's next 32 records lie: one division each
    long long where = -1;
    {
      const int r = r0 + kWeighWarps * lane;
      if (r < rec1) {
        const int page = r / page_recs;
        const long long block = __ldg(table + page);
        if (block >= 0 && block < p.num_blocks) where = (block * p.Hkv + h) * page_recs + (r - page * page_recs);
        else if (!kWeigh) atomicOr(p.err, PE_ERR_BLOCK_RANGE);
      }
    }
    const int n = min(32, (rec1 - r0 + kWeighWarps - 1) / kWeighWarps);
    const uint32_t live = __ballot_sync(0xffffffffu, where >= 0);  // (the first n lanes' at most)
    using W = WeighShared<D, kTiles>;
    // lanes send for their own records: of [i, i + 2)
    auto send = [&](int i, int many) {
      if (lane >= i && lane < min(i + many, n) && where >= 0) {
        const uint32_t at = turn + lane;
        uint64_t* bar = &sh.bars[warp][at % kStages];
        uint8_t* to = sh.ring[warp][at % kStages];
        const uint8_t* rec = p.cache + where * Record<D>::kBytes;
        mbar_arrive_expect_tx(bar, W::kCodes + W::kScales);
        bulk_load(to, rec + Record<D>::kK, W::kCodes, bar);
        bulk_load(to + W::kCodes, rec + Record<D>::kKs, W::kScales, bar);
      }
    };
    auto old_of = [&](int i) {  // what this lane's key of record i had
      const int row = g + 8 * (lane & 3), j = 16 * (r0 + kWeighWarps * i) + row;
      const long long at = __shfl_sync(0xffffffffu, where, i) * 16 + row;
      float v = 0.f;
      if (row < 16 && j < reach && (live >> i & 1)) {
        if (more) v = p.out[at];
        else if (p.mass && j < fresh) v = p.mass[at];
      }
      return v;
    };
    send(0, 2);
    float old = kWeigh ? old_of(0) : 0.f;
    for (int i = 0; i < n; ++i) {
      const uint32_t at = turn + i;
      if ((i & 1) == 0) {
        __syncwarp();  // (the stages that come next have been read)
        send(i + 2, 2);
      }
      const float old0 = old;
      if (kWeigh && i + 1 < n) old = old_of(i + 1);
      if (!(live >> i & 1)) {
        // (its stage was not used: it counts as done)
        if (lane == 0) mbar_arrive_expect_tx(&sh.bars[warp][at % kStages], 0);
        __syncwarp();
        (void)mbar_wait(&sh.bars[warp][at % kStages], (at / kStages) & 1);
        continue;
      }
      const int j0 = 16 * (r0 + kWeighWarps * i);
      if (!mbar_wait(&sh.bars[warp][at % kStages], (at / kStages) & 1)) {
        atomicOr(p.err, PE_ERR_TIMEOUT);
        (void)mbar_wait(&sh.bars[warp][at % kStages], (at / kStages) & 1);
      }
      uint32_t a[D / 16][4];
      {
        KeyWords<D> words;
        words.load(sh.ring[warp][at % kStages], lane);
        words.convert(a);
      }
      const long long cur = kWeigh ? __shfl_sync(0xffffffffu, where, i) : 0;
      const int row = g + 8 * (lane & 3);  // (lanes with row >= 16 have none to write)
      const bool first = track || (r0 == rec0 + warp && i == 0);
      float2 w = make_float2(0.f, 0.f), w2 = w;  // of rows g and g + 8
      // kSlow: a record at which some column ends, or from which the sums' bases are taken
      auto tile = [&](int x, float2& sum, auto slow) {
        constexpr bool kSlow = decltype(slow)::value;
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
          const uint4 q = kTiles == 1 ? q1[s] : sh.q[x][s][lane];
          mma_f16(d, a[2 * s], q.x, q.y);
          mma_f16(d, a[2 * s + 1], q.z, q.w);
        }
        const float2 f = *reinterpret_cast<const float2*>(&sh.factor[8 * x + t2]);
        // (scores are rounded once, before the differences: from a fused one a large score's
        // rounding would come back as an exponent)
        mul2(d[0], d[1], f, zero);
        mul2(d[2], d[3], f, zero);
        if (kSlow) {
          const int2 lim = *reinterpret_cast<const int2*>(&sh.limit[8 * x + t2]);
          if (j0 + g >= lim.x) d[0] = -INFINITY;
          if (j0 + g >= lim.y) d[1] = -INFINITY;
          if (j0 + g + 8 >= lim.x) d[2] = -INFINITY;
          if (j0 + g + 8 >= lim.y) d[3] = -INFINITY;
        }
        if (kWeigh) {
          const float2 z = *reinterpret_cast<const float2*>(&sh.lse[8 * x + t2]);  // (negative: -lse)
          const float2 p0 = add2(d[0], d[1], z), p1 = add2(d[2], d[3], z);
          sum = add2(sum.x, sum.y, make_float2(exp2_approx(p0.x) + exp2_approx(p0.y), exp2_approx(p1.x) + exp2_approx(p1.y)));
        } else {
          if (kSlow && first) {
            const float m0 = fmaxf(st.m[x][0], fmaxf(d[0], d[2])), m1 = fmaxf(st.m[x][1], fmaxf(d[1], d[3]));
            st.l[x][0] *= exp2_approx(st.m[x][0] - m0);
            st.l[x][1] *= exp2_approx(st.m[x][1] - m1);
            st.m[x][0] = m0;
            st.m[x][1] = m1;
          }
          const float2 low = make_float2(-st.m[x][0], -st.m[x][1]);
          const float2 p0 = add2(d[0], d[1], low), p1 = add2(d[2], d[3], low);
          st.l[x][0] += exp2_approx(p0.x) + exp2_approx(p1.x);
          st.l[x][1] += exp2_approx(p0.y) + exp2_approx(p1.y);
        }
      };
      // (two tiles between branches, for their products to overlap)
      auto all_tiles = [&](auto slow) {
        if (kTiles == 1) {
          tile(0, w, slow);
        } else {
#pragma unroll
          for (int x = 0; x < kTiles; x += 2) {
            if (x >= tiles) break;
            tile(x, w, slow);
            tile(x + 1, w2, slow);
          }
        }
      };
      if (j0 + 16 > sh.least || (!kWeigh && first)) all_tiles(std::true_type());
      else all_tiles(std::false_type());
      float w0 = w.x + w2.x, w1 = w.y + w2.y;
      if (kWeigh) {
        w0 += __shfl_xor_sync(0xffffffffu, w0, 1);
        w1 += __shfl_xor_sync(0xffffffffu, w1, 1);
        w0 += __shfl_xor_sync(0xffffffffu, w0, 2);
        w1 += __shfl_xor_sync(0xffffffffu, w1, 2);
        if (row < 16 && j0 + row < reach) p.out[cur * 16 + row] = old0 + ((lane & 3) ? w1 : w0);
      }
    }
    turn += n;
    __syncwarp();
  }
}

__device__ __forceinline__ float2 merge(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  return make_float2(m, a.y * (a.x == m ? 1.f : exp2_approx(a.x - m)) + b.y * (b.x == m ? 1.f : exp2_approx(b.x - m)));
}

// The columns' pairs over the CTA's lanes and warps, into sh.sums.
template <int D, int kTiles>
__device__ __forceinline__ void join_stats(WeighShared<D, kTiles>& sh, int tiles, const Stats<kTiles>& st) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    if (kTiles > 1 && i >= tiles) break;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float2 v = make_float2(st.m[i][c], st.l[i][c]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
        v = merge(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
      if ((lane >> 2) == 0) sh.join[warp][8 * i + 2 * (lane & 3) + c] = v;
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 8 * tiles; c += kWeighThreads) {
    float2 v = sh.join[0][c];
#pragma unroll
    for (int w = 1; w < kWeighWarps; ++w) v = merge(v, sh.join[w][c]);
    sh.sums[c] = v;
  }
}
template <int D, int kTiles>
__device__ __forceinline__ void statistics(const WeighParams& p, WeighShared<D, kTiles>& sh, int b, int h, int rec0, int rec1,
                                           int reach, int n, uint32_t& turn, Stats<kTiles>& st) {
  const int tiles = (n + 7) >> 3;
#pragma unroll 1
  for (int track = 0; track < 2; ++track) {
    st.clear();
    sweep<D, kTiles, false>(p, sh, b, h, rec0, rec1, reach, tiles, false, track, turn, st);
    join_stats<D, kTiles>(sh, tiles, st);
    bool large = false;
    for (int c = threadIdx.x; c < n; c += kWeighThreads) large |= !(sh.sums[c].y <= 0x1p100f);  // (infinite ones may have become NaN)
    if (!__syncthreads_or(large)) break;
  }
}
__device__ __forceinline__ float log_sum(float2 v) { return v.y == 0.f ? INFINITY : v.x + log2f(v.y); }

// Rows of the request, and how far they reach (nothing: no keys); columns of a key head.
template <int D, int kTiles>
__device__ __forceinline__ int request_reach(const WeighParams& p, WeighShared<D, kTiles>& sh, int b, bool report, int& r0, int& columns) {
  int r1;
  request_rows(p, b, r0, r1);
  if (threadIdx.x == 0) sh.reach = 0;
  if (threadIdx.x < kWeighWarps * kStages) {
    mbar_init(&sh.bars[0][0] + threadIdx.x, 1);
    mbar_init_fence();
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  int most = 0;
  if (r1 - r0 <= kLiveRows) {
    if (threadIdx.x < 32) {
      int n = 0;
      for (int t0 = r0; t0 < r1; t0 += 32) {
        const int limit = t0 + lane < r1 ? row_limit(p, t0 + lane, report) : 0;
        const uint32_t m = __ballot_sync(0xffffffffu, limit > 0);
        if (limit > 0) sh.rows[n + __popc(m & ((1u << lane) - 1))] = t0 + lane;
        n += __popc(m);
        most = max(most, limit);
      }
      if (lane == 0) sh.live = n;
    }
  } else {
    for (int t = r0 + threadIdx.x; t < r1; t += kWeighThreads) most = max(most, row_limit(p, t, report));
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0 && most) atomicMax(&sh.reach, most);
  __syncthreads();
  columns = (r1 - r0 <= kLiveRows ? sh.live : r1 - r0) * p.G;
  if (r1 - r0 > kLiveRows && threadIdx.x == 0) sh.live = 0;  // (all rows)
  __syncthreads();
  return sh.reach;
}

// Both looks in one kernel: a cluster per request and key head, the columns' sums
// exchanged in between; the second look finds the keys in L2 (some 40 clusters at once, of
// 2.4 MB of keys each at 32,000 keys of 128).
template <int D, int kTiles>
__global__ void __launch_bounds__(kWeighThreads, 2) weigh_pair_kernel(const WeighParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  WeighShared<D, kTiles>& sh = *reinterpret_cast<WeighShared<D, kTiles>*>(smem);
  const int C = p.chunks, rank = (int)cluster_rank();
  const int pair = blockIdx.x / C, b = pair / p.Hkv, h = pair - b * p.Hkv;
  if (p.offsets && !offsets_valid(p.offsets, p.B, p.T, 0)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.err, PE_ERR_OFFSETS);
    return;
  }
  int r0, columns;
  const int reach = request_reach(p, sh, b, h == 0 && rank == 0, r0, columns);
  if (reach == 0) return;
  const int recs = (reach + 15) >> 4, per = (recs + C - 1) / C;
  const int rec0 = min(recs, rank * per), rec1 = min(recs, rec0 + per);
  const bool listed = sh.live > 0;
  uint32_t turn = 0;  // of the warp's ring
  for (int c0 = 0; c0 < columns; c0 += 8 * kTiles) {
    const int n = min(8 * kTiles, columns - c0), tiles = (n + 7) >> 3;
    load_columns(p, sh, r0, listed, h, c0, n);
    Stats<kTiles> st;
    statistics<D, kTiles>(p, sh, b, h, rec0, rec1, reach, n, turn, st);
    __syncwarp();
    cluster_sync();
    for (int c = threadIdx.x; c < n; c += kWeighThreads) {
      float2 v = *at_rank(&sh.sums[c], 0);
      for (int r = 1; r < C; ++r) v = merge(v, *at_rank(&sh.sums[c], r));
      sh.lse[c] = sh.limit[c] ? -log_sum(v) : -INFINITY;
    }
    cluster_sync();  // (the sums have been read)
    __syncthreads();
    sweep<D, kTiles, true>(p, sh, b, h, rec0, rec1, reach, tiles, c0 > 0, false, turn, st);
  }
}

// The two looks as kernels of their own, a CTA per chunk of keys: where there are too few
// pairs of request and key head for the clusters to fill the GPU.
template <int D, int kTiles, bool kWeigh>
__global__ void __launch_bounds__(kWeighThreads, kTiles == 1 ? 4 : 2) weigh_chunk_kernel(const WeighParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  WeighShared<D, kTiles>& sh = *reinterpret_cast<WeighShared<D, kTiles>*>(smem);
  const int b = blockIdx.y / p.Hkv, h = blockIdx.y - b * p.Hkv;
  int r0, columns;
  const int reach = request_reach(p, sh, b, !kWeigh && h == 0 && blockIdx.x == 0, r0, columns);
  if (kWeigh) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (__ldcg(p.lse + (long long)p.T * p.Hq) != 0.f) return;  // offsets no partition
  }
  const int rec0 = blockIdx.x * (p.chunk >> 4), rec1 = min((reach + 15) >> 4, rec0 + (p.chunk >> 4));
  if (rec0 >= rec1) return;
  const bool listed = sh.live > 0;
  uint32_t turn = 0;  // of the warp's ring
  for (int c0 = 0; c0 < columns; c0 += 8 * kTiles) {
    const int n = min(8 * kTiles, columns - c0), tiles = (n + 7) >> 3;
    load_columns(p, sh, r0, listed, h, c0, n);
    Stats<kTiles> st;
    if (!kWeigh) {
      statistics<D, kTiles>(p, sh, b, h, rec0, rec1, reach, n, turn, st);
      __syncthreads();
    }
    for (int c = threadIdx.x; c < n; c += kWeighThreads) {
      const int of = (c0 + c) / p.G;
      const long long at = (long long)(listed ? sh.rows[of] : r0 + of) * p.Hq + h * p.G + (c0 + c) % p.G;
      if (kWeigh) sh.lse[c] = -__ldcg(p.lse + at);
      else p.parts[(long long)blockIdx.x * p.T * p.Hq + at] = sh.sums[c];
    }
    if (kWeigh) {
      __syncthreads();
      sweep<D, kTiles, true>(p, sh, b, h, rec0, rec1, reach, tiles, c0 > 0, false, turn, st);
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
  float2 v = make_float2(kLowest, 0.f);
  for (int c = 0; c < n; ++c) v = merge(v, __ldcg(p.parts + (long long)c * p.T * p.Hq + i));
  p.lse[i] = log_sum(v);
}

}  // namespace pe

namespace {

// Keys of a chunk: as many as keep the GPU in work with `want` chunks.  With one tile of columns a
// chunk costs little to begin with; with more it loads and converts all of them.
int weigh_chunk(int B, int Hkv, int64_t keys, int want) {
  int chunk = 4096;
  while (chunk > 128 && (int64_t)B * Hkv * ((keys + chunk - 1) / chunk) < want) chunk /= 2;
  return chunk;
}

// Little work: pairs, one launch (one token over 4000 keys of 8 heads 14 us; three launches 19).
// Else one tile of columns: chunks (b256 tokens 1.18 ms; the pair kernel 1.38, at its 128 registers);
// more: pairs, where these fill the GPU (b64 drafts 0.77 ms).
template <int D, int kTiles>
int weigh(pe::WeighParams p, int sms, cudaStream_t st) {
  constexpr int kSmem = (int)sizeof(pe::WeighShared<D, kTiles>);
  static std::atomic<unsigned long long> done[3];
  const int64_t keys = (int64_t)p.bt_width * p.block_size, pairs = (int64_t)p.B * p.Hkv;
  const bool small = pairs * keys <= (int64_t)sms * 2048;
  if (small || (kTiles > 1 && pairs * 4 >= sms / 2)) {
    auto kernel = pe::weigh_pair_kernel<D, kTiles>;
    if (!pe_host::allow_smem(kernel, kSmem, done[0])) return PE_ECUDA;
    p.chunks = 1;  // CTAs of a cluster: up to four (b64 drafts 1.46 ms with eight, 1.35 with four at the time)
    while (p.chunks < 4 && keys > 1024 * p.chunks) p.chunks *= 2;
    while (small && p.chunks < 16 && pairs * p.chunks * 2 <= sms && keys > 256 * p.chunks) p.chunks *= 2;
    static std::atomic<unsigned long long> wide{0};
    if (p.chunks > 8 && !pe_host::allow_wide_clusters(kernel, wide)) return PE_ECUDA;
    const cudaError_t rc = pe_host::launch_clusters(kernel, dim3((unsigned)(pairs * p.chunks)), pe::kWeighThreads, p.chunks, kSmem,
                                                    false, st, p);
    return rc == cudaSuccess ? pe_host::launch_status() : PE_ECUDA;
  }
  auto stats = pe::weigh_chunk_kernel<D, kTiles, false>;
  auto weigh = pe::weigh_chunk_kernel<D, kTiles, true>;
  if (!pe_host::allow_smem(stats, kSmem, done[1]) || !pe_host::allow_smem(weigh, kSmem, done[2])) return PE_ECUDA;
  const dim3 grid(p.chunks, p.B * p.Hkv);
  stats<<<grid, pe::kWeighThreads, kSmem, st>>>(p);
  // the other two may start while the one before drains, and wait in the kernel for it
  const unsigned cols = (unsigned)(((int64_t)p.T * p.Hq + pe::kWeighThreads - 1) / pe::kWeighThreads);
  cudaError_t rc = pe_host::launch_clusters(pe::weigh_join_kernel, dim3(cols), pe::kWeighThreads, 1, 0, true, st, p);
  if (rc == cudaSuccess) rc = pe_host::launch_clusters(weigh, grid, pe::kWeighThreads, 1, kSmem, true, st, p);
  return rc == cudaSuccess ? pe_host::launch_status() : PE_ECUDA;
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
  // columns of a request that has its even share of the rows
  const int64_t columns = ((int64_t)a->T + a->B - 1) / a->B * p.G;
  p.chunk = weigh_chunk(a->B, a->Hkv, keys, columns <= 8 ? 4096 : 256);
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
  pe_host::DeviceInfo dev;
  if (pe_host::device_info(&dev) != PE_OK) return PE_ECUDA;
  if (a->D == 64)
    return columns <= 8 ? weigh<64, 1>(p, dev.sm_count, st) : columns <= 32 ? weigh<64, 4>(p, dev.sm_count, st) : weigh<64, 16>(p, dev.sm_count, st);
  return columns <= 8 ? weigh<128, 1>(p, dev.sm_count, st) : columns <= 32 ? weigh<128, 4>(p, dev.sm_count, st) : weigh<128, 16>(p, dev.sm_count, st);
}

}  // extern "C"
