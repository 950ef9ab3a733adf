// Sampling from filtered logits rows (pe_draft_sample) and rejection sampling
// against filtered distributions (pe_verify_filtered).  Definitions and the
// row's arithmetic: pe_filter.cuh.
//
// filter_kernel: a cluster of C CTAs per row, each with a slice of it in shared
// memory.
//  1. Every thread takes the maximum of its columns.
//  2. A value that every kept column reaches: under a top-k of at most kListK the k-th
//     largest of the thread maxima; under top-p, where the columns of at least 2^-8 or 2^-12 of
//     the largest weight hold the share, that weight, else what the last kept column weighs at
//     least; under min-p its floor.  The columns from there on go to a list in CTA 0's shared
//     memory, the other CTAs leave, and CTA 0 finds rank, preceding weight and draw: up to kPairs
//     columns by comparing all pairs, up to kListCap by bins.
//  3. Where the list does not do (a larger k, more columns than it holds, ties), a histogram over
//     the whole row shows between which values the cut lies, the weight above is added up, and the
//     columns between are listed; failing that (ties), the cut's value is found bit by bit.
//  4. The draw from many columns: the CTAs' kept weights are exchanged, and the CTA, the warp and
//     the vector in whose share the draw falls look for the column.
//
// 1792 rows of 151936 bf16 columns, read once (81 us at the copy rate): greedy 182 us, top-k 20 216,
// top-p 0.95 395, unfiltered 349.  What bounds them is the time that a row's slices stay in
// shared memory: some 3,500 clocks until they have landed, then a chain of barriers and short steps
// (top-k 20: 14,000 clocks, 21,000 in CTA 0); four CTAs of 256 threads on an SM overlap them.
// Of that chain: a CTA barrier takes 50 clocks, a cluster barrier with a remote store 1,100.
// Measured and left: CTAs of 512 threads, two on an SM (top-k 20 465 us; the step to
// four of 256, with wider clusters and the histogram, 399); 64-bit arithmetic in every thread (1792 mixed
// rows 841 us, 614 by the end of the step that took it out).
// Verification of 256 such requests: 618 us, of which this kernel 570.
// residual_kernel: a cluster per request finds the first rejection and draws
// from max(0, p - q).
#include "pe_filter.cuh"

namespace pe {

struct FilterParams {
  const char* rows_a;  // target rows, or the only ones
  const char* rows_b;  // draft rows
  long long a_bytes, b_bytes;
  int V, nvec, per_cta, seg, n, na, C;
  int Kp;                     // verification: rows of a request - 1
  int per;                    // sampling: rows that share parameters
  int src_rows;
  const int32_t* sample_idx;  // or NULL
  AskedArrays asked;
  const float* u;
  // sampling
  int32_t* out_tokens;
  float* out_prob;
  // verification
  const int32_t* tokens;
  const float* coins;
  int32_t* accepted;
  int32_t* bonus;
  float* chance;
  RowCut* cuts;  // [n]
  Kept* kept;    // [na][kKeptCap]
  uint32_t* err;
};

constexpr int kListBins = 256;
constexpr int kSteps = 4 * kFT;   // bins of the search for a cut over the whole row

struct FilterShared {
  uint64_t bars[kFW];
  unsigned long long sums[2][kMaxCluster];  // exchanged by the CTAs, in turns
  unsigned long long warp_sum[kFW], warp_large[2][kFW];
  unsigned long long large[2][kMaxCluster];
  uint32_t counts[2][kMaxCluster];
  uint32_t warp_count[kFW];
  uint32_t maxima[kMaxCluster], bounds[kMaxCluster], shares[kMaxCluster];
  unsigned long long total, above;
  uint32_t own, bin, in_bin, stored;
  uint32_t cut_key;
  int cut_tie, tie;
  float2 table[32];
  double wx;
  Rates rates;
  float2 inverse[2];
  float floor;
  int first;
  uint32_t hist[kFT];
  unsigned short hits[kFW][64];
  union alignas(16) {
    unsigned long long list[kListCap];         // candidates: (value's key, ~column)
    uint32_t steps[kSteps];
  };
};
// In the place of CTA 0's slice, once the list holds all that is needed of it.
constexpr int kPairs = kFT;  // columns of a list that is resolved by comparing all pairs
struct FilterLists {
  struct {  // the columns of one bin (pairs: of the list)
    unsigned long long key[kListCap];
    unsigned long long w[kListCap];
  } sel;
  unsigned long long mass[kListBins];
  uint32_t count[kListBins];
};

__device__ __forceinline__ unsigned long long warp_sum_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ uint32_t key_of(unsigned long long k) { return (uint32_t)(k >> 32); }

// A CTA's view of its row.
template <int DT>
struct Slice {
  const uint4* v;    // the slice in shared memory
  int n, lo, hi;     // vectors of the slice; of this warp's segment
  int col0;          // column of the slice's first element
  int lane, warp, rank, C;
  FilterShared* sh;
  int turn;          // exchanges so far

  // Sum over the cluster of one count and one weight (given by every thread of the CTA
  // as its warp's: lane 0's values count).
  __device__ __forceinline__ void exchange(uint32_t& count, unsigned long long& sum,
                                           unsigned long long* before = nullptr, uint32_t* count_before = nullptr) {
    cta_sync();  // the arrays' last readers
    if (lane == 0) {
      sh->warp_count[warp] = count;
      sh->warp_sum[warp] = sum;
    }
    cta_sync();
    const int t = threadIdx.x;
    const int slot = turn & 1;
    if (t < C) {
      uint32_t c = 0;
      unsigned long long s = 0;
      for (int w = 0; w < kFW; ++w) {
        c += sh->warp_count[w];
        s += sh->warp_sum[w];
      }
      *at_rank(&sh->counts[slot][rank], t) = c;
      *at_rank(&sh->sums[slot][rank], t) = s;
    }
    cluster_sync();
    ++turn;
    count = 0;
    sum = 0;
    for (int r = 0; r < C; ++r) {
      if (before && r == rank) {
        *before = sum;
        *count_before = count;
      }
      count += sh->counts[slot][r];
      sum += sh->sums[slot][r];
    }
  }

  // The warp's share of the row's weight.  Vectors of small weights (pe_filter.cuh) are added up as
  // they come, a vector at a time: a sum whose last bit is 2^-23, and what that drops.  The others
  // are queued (a branch in the loop would be taken by one lane or another nearly every time)
  // and weighed in full, an element a lane.  large: the share of the columns of at least 2^-12 of the largest weight.
  __device__ __forceinline__ unsigned long long mass(const Scale& sc, unsigned long long (&large)[2]) {
    const float big = sc.inf ? -INFINITY : sc.M - 16.f * sc.octave, top8 = sc.inf ? sc.M : sc.M - 8.f * sc.octave,
                top12 = sc.inf ? sc.M : sc.M - 12.f * sc.octave;
    ShortSum<1> small;
    ShortSum<256> to8, to12;  // (for a choice with a margin)
    WeightSum<256> all;
    uint32_t queued = 0;
    auto take = [&]() {  // an element a lane: a large vector has one or two large ones
      __syncwarp();
      for (uint32_t j0 = 0; j0 < queued; j0 += 32 / Elt<DT>::kN) {
        const uint32_t j = j0 + lane / Elt<DT>::kN;
        if (j < queued) {
          const float x = Elt<DT>::element(v, sh->hits[warp][j], lane % Elt<DT>::kN);
          const float2 w = weight(sc, sh->table, x);
          all.add(w.x, w.y);
          if (x >= top8) to8.add(w.x + w.y);
          else if (x >= top12) to12.add(w.x + w.y);
        }
      }
      queued = 0;
      __syncwarp();
    };
    auto look = [&](bool clean) {
      small = ShortSum<1>();
#pragma unroll 2
      for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + lane;
        bool put = false;
        if (i < hi) {
          const uint4 q = v[i];
          put = Elt<DT>::max_of(q) >= big;
          if (!put) {
            float2 sum = make_float2(0.f, 0.f), rest = sum;
#pragma unroll
            for (int e = 0; e < Elt<DT>::kN; e += 2)
              add_small<DT>(sc, make_float2(Elt<DT>::get(q, e), Elt<DT>::get(q, e + 1)), clean, sum, rest);
            if (DT == PE_F32) sum = fma2(rest, make_float2(0.693147181f, 0.693147181f), sum);
            small.add(sum.x + sum.y);
          }
        }
        if (clean) continue;
        const uint32_t m = __ballot_sync(0xffffffffu, put);
        if (m) {
          if (put) sh->hits[warp][queued + __popc(m & ((1u << lane) - 1))] = (unsigned short)i;
          queued += __popc(m);
          if (queued > 32) take();  // (room for another 32 is needed)
        }
      }
    };
    look(false);
    take();
    if (DT == PE_BF16 && __any_sync(0xffffffffu, small.lo != small.lo)) look(true);
    const unsigned long long at8 = to8.fixed(kSumBits);
    large[0] = warp_sum_u64(at8);
    large[1] = warp_sum_u64(at8 + to12.fixed(kSumBits));
    small.lo = fmaf(kSmallMean, (small.s - 1.f) + small.lo, small.lo);
    return warp_sum_u64(all.fixed(kSumBits) + small.fixed(kSumBits));
  }

  // The warp's share of the weight that a cut keeps.
  __device__ __forceinline__ unsigned long long kept_mass(const Scale& sc, const Cut& cut) {
    WeightSum<256> ws;
    for (int i = lo + lane; i < hi; i += 32) {
      const uint4 q = v[i];
      if (value_key(Elt<DT>::max_of(q)) < cut.key) continue;
#pragma unroll
      for (int e = 0; e < Elt<DT>::kN; ++e) {
        const float x = Elt<DT>::get(q, e);
        if (cut.keeps(x, col0 + i * Elt<DT>::kN + e)) {
          const float2 w = weight(sc, sh->table, x);
          ws.add(w.x, w.y);
        }
      }
    }
    return warp_sum_u64(ws.fixed(kSumBits));
  }

  // Columns with key >= t: how many, and (kMass) their weight.
  template <bool kMass>
  __device__ __forceinline__ void above(const Scale& sc, uint32_t t, uint32_t& count, unsigned long long& sum) {
    uint32_t c = 0;
    WeightSum<256> ws;
    for (int i = lo + lane; i < hi; i += 32) {
      const uint4 q = v[i];
#pragma unroll
      for (int e = 0; e < Elt<DT>::kN; ++e) {
        const float x = Elt<DT>::get(q, e);
        if (value_key(x) >= t) {
          ++c;
          if (kMass) {
            const float2 w = weight(sc, sh->table, x);
            ws.add(w.x, w.y);
          }
        }
      }
    }
    count = __reduce_add_sync(0xffffffffu, c);
    sum = kMass ? warp_sum_u64(ws.fixed(kSumBits)) : 0ull;
    exchange(count, sum);
  }

  // The largest value whose columns from it on number at least k (kMass: weigh at least `target`).
  template <bool kMass>
  __device__ __forceinline__ uint32_t search(const Scale& sc, uint32_t k, double target) {
    uint32_t t = 0;
    for (int bit = 31; bit >= 32 - Elt<DT>::kKeyBits; --bit) {
      const uint32_t trial = t | (1u << bit);
      uint32_t c;
      unsigned long long s;
      above<kMass>(sc, trial, c, s);
      if (kMass ? (double)s >= target : c >= k) t = trial;
    }
    if (Elt<DT>::kKeyBits == 16 && !(t >> 31)) t |= 0xffffu;  // (a negative bf16's low bits)
    return t;
  }

  // The columns between which a cut lies, by one pass with a histogram: `steps` bins of
  // x from M down to where weights are 2^-octaves, taken from the columns that `cut` keeps,
  // of counts or of weights (relative to the bin, in 13 bits: a bin's error is far below the
  // margins).  Afterwards every kept column of at least `hi` belongs to the wanted prefix, of
  // `count` columns; none below `lo` does.  False: the range does not reach the target.
  template <bool kMass>
  __device__ __forceinline__ bool steer(const Scale& sc, const Cut& cut, float octaves, double target, uint32_t* steps, float& lo_x,
                                        float& hi_x) {
    const int tid = threadIdx.x;
    const float width = octaves / (float)kSteps, range = octaves * sc.octave, per = (float)kSteps / range;
    for (int i = tid; i < kSteps; i += kFT) steps[i] = 0;
    cta_sync();
    for (int i = lo + lane; i < hi; i += 32) {
      const uint4 q = v[i];
      if (Elt<DT>::max_of(q) <= sc.M - range) continue;
#pragma unroll
      for (int e = 0; e < Elt<DT>::kN; ++e) {
        const float x = Elt<DT>::get(q, e);
        const float d = sc.M - x;
        if (d < range && cut.keeps(x, col0 + i * Elt<DT>::kN + e)) {
          const int bin = min((int)(d * per), kSteps - 1);
          uint32_t one = 1;
          if (kMass) {
            float w;
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"((float)(bin + 1) * width - d * sc.ch));
            one = (uint32_t)(w * 4096.f);
          }
          atomicAdd(&steps[bin], one);
        }
      }
    }
    cluster_sync();
    // every CTA adds up all of them: the same answer everywhere
    double c[4], mine = 0.0;
    uint32_t sum[4] = {0, 0, 0, 0};
    for (int r = 0; r < C; ++r) {
      const uint4 q = *reinterpret_cast<const uint4*>(at_rank(steps, r) + 4 * tid);
      sum[0] += q.x, sum[1] += q.y, sum[2] += q.z, sum[3] += q.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = kMass ? (double)sum[i] * (double)exp2f(-(float)(4 * tid + i + 1) * width) * (1.0 / 4096) : (double)sum[i];
      mine += c[i];
    }
    double pre = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double x = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += x;
    }
    cta_sync();
    double* part = reinterpret_cast<double*>(sh->warp_sum);
    if (lane == 31) part[warp] = pre;
    if (tid == 0) sh->bin = kSteps, sh->in_bin = kSteps;
    cta_sync();
    pre -= mine;
    for (int w = 0; w < warp; ++w) pre += part[w];
    const double slack = kMass ? target * 0x1p-11 : 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double next = pre + c[i];
      // the cut lies here at the earliest, or there at the latest (atomics: two threads' roundings
      // may both claim it, and every CTA has to take the same)
      if (pre < target - slack && next >= target - slack) atomicMin(&sh->bin, (uint32_t)(4 * tid + i));
      if (pre < target + slack && next >= target + slack) atomicMin(&sh->in_bin, (uint32_t)(4 * tid + i));
      pre = next;
    }
    cluster_sync();  // (the histograms have been read)
    const int first = (int)sh->bin, last = (int)sh->in_bin;
    if (last >= kSteps) return false;
    // edges of the bins as the conversion above sees them: lowered and raised by its rounding
    const float eps = 0x1p-21f * (range + fabsf(sc.M));
    hi_x = first ? sc.M - (float)first / per + eps : INFINITY;
    lo_x = sc.M - (float)(last + 1) / per - eps;
    return true;
  }

  // Column of the r-th (from 1) of the columns of value `key`.
  __device__ __forceinline__ int nth_tie(uint32_t key, uint32_t r) {
    uint32_t c = 0;
    for (int i = lo + lane; i < hi; i += 32) {
      const uint4 q = v[i];
#pragma unroll
      for (int e = 0; e < Elt<DT>::kN; ++e) c += value_key(Elt<DT>::get(q, e)) == key;
    }
    c = __reduce_add_sync(0xffffffffu, c);
    uint32_t all = c, before = 0;
    unsigned long long none = 0, none_before;
    exchange(all, none, &none_before, &before);
    for (int w = 0; w < warp; ++w) before += sh->warp_count[w];
    if (before < r && r <= before + c) {  // in this warp's segment
      uint32_t at = before;
      for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + lane;
        uint32_t mine = 0;
        const uint4 q = v[min(i, hi - 1)];
        if (i < hi) {
#pragma unroll
          for (int e = 0; e < Elt<DT>::kN; ++e) mine += value_key(Elt<DT>::get(q, e)) == key;
        }
        uint32_t pre = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t x = __shfl_up_sync(0xffffffffu, pre, o);
          if (lane >= o) pre += x;
        }
        if (at + pre - mine < r && r <= at + pre) {
          uint32_t left = r - (at + pre - mine);
#pragma unroll
          for (int e = 0; e < Elt<DT>::kN; ++e)
            if (value_key(Elt<DT>::get(q, e)) == key && --left == 0) {
              const int col = col0 + i * Elt<DT>::kN + e;
              for (int t = 0; t < C; ++t) *at_rank(&sh->tie, t) = col;
            }
        }
        at += __shfl_sync(0xffffffffu, pre, 31);
      }
    }
    cluster_sync();
    return r > all ? INT32_MAX : sh->tie;
  }
};

// The column (relative to the slice) in a warp's segment [lo, hi) of vectors where
// the running sum passes `target`; get(i, from, to, sum) adds columns from..to-1 of vector
// i to a sum.  Should roundings leave none, the last column that weighs anything; where every
// vector by itself rounds to nothing (a warp's share adds up what its vectors' roundings drop),
// the first column of any weight.  -1: there is none.  All lanes return it.
template <int kN, int kBias, class F>
__device__ __forceinline__ int find_column(int lo, int hi, int lane, unsigned long long target, int bits, const F& get) {
  unsigned long long at = 0;
  int found = -1;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    unsigned long long mine = 0;
    if (i < hi) {
      WeightSum<kBias> ws;
      get(i, 0, kN, ws);
      mine = ws.fixed(bits);
    }
    unsigned long long pre = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long x = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += x;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, at + pre > target);
    const uint32_t some = __ballot_sync(0xffffffffu, mine > 0);
    const int src = hit ? __ffs(hit) - 1 : some ? 31 - __clz(some) : -1;
    if (src >= 0) {
      int col = -1;
      if (lane == src) {
        WeightSum<kBias> upto;
        unsigned long long last = 0;
        for (int e = 0; e < kN; ++e) {
          get(i, e, e + 1, upto);
          const unsigned long long now = upto.fixed(bits);
          if (now > last) col = i * kN + e;
          last = now;
          if (at + (pre - mine) + now > target) break;
        }
      }
      found = __shfl_sync(0xffffffffu, col, src);
      if (hit) return found;
    }
    at += __shfl_sync(0xffffffffu, pre, 31);
  }
  if (found >= 0) return found;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    int first = -1;
    for (int e = kN - 1; e >= 0 && i < hi; --e) {
      WeightSum<kBias> one;
      get(i, e, e + 1, one);
      if (one.positive()) first = i * kN + e;
    }
    const uint32_t some = __ballot_sync(0xffffffffu, first >= 0);
    if (some) return __shfl_sync(0xffffffffu, first, __ffs(some) - 1);
  }
  return -1;
}

// After an exchange of the warps' shares: in the CTA in whose share `at` falls, all warps
// take a part of the segment of the warp in whose share it falls (`weigh` gives a part's weight);
// the warp whose part it is, or -1 in the other CTAs.  pre: the weight before that part.  Parts are
// rounded by themselves: where all of them round to nothing, one warp takes the whole segment.
template <int DT, class F>
__device__ __forceinline__ int narrow(Slice<DT>& s, FilterShared& sh, int seg, int v_lo, int v_hi, unsigned long long at,
                                      unsigned long long before, unsigned long long& pre, const F& weigh) {
  int owner = -1;
  pre = before;
  for (int w = 0; w < kFW; ++w) {
    const unsigned long long next = pre + sh.warp_sum[w];
    if (pre <= at && at < next) {
      owner = w;
      before = pre;
    }
    pre = next;
  }
  if (owner < 0) return -1;  // (the same in all threads of the CTA)
  const int o_lo = min(v_hi, v_lo + owner * seg), o_hi = min(v_hi, o_lo + seg), sub = (o_hi - o_lo + kFW - 1) / kFW;
  s.lo = min(o_hi, o_lo + s.warp * sub);
  s.hi = min(o_hi, s.lo + sub);
  const unsigned long long mine = weigh();
  cta_sync();
  if (s.lane == 0) sh.warp_sum[s.warp] = mine;
  cta_sync();
  int chosen = kFW - 1;  // (roundings may leave the last part that weighs anything)
  while (chosen >= 0 && sh.warp_sum[chosen] == 0) --chosen;
  pre = before;
  if (chosen < 0) {
    s.lo = o_lo;
    s.hi = o_hi;
    return 0;
  }
  for (int w = 0; w < chosen; ++w) {
    if (at < pre + sh.warp_sum[w]) {
      chosen = w;
      break;
    }
    pre += sh.warp_sum[w];
  }
  return chosen;
}

// Largest key prefix (upper 16 bits) that at least k of the CTA's threads reach: by a
// histogram of the distance from the largest one, or bit by bit where that is short.
// hist is zero before and after.
__device__ __forceinline__ uint32_t kth_prefix(uint32_t* hist, uint32_t mine, uint32_t top, uint32_t k) {
  const uint32_t d = top - mine;
  if (d < kFT) atomicAdd(&hist[d], 1u);
  cta_sync();
  // every warp adds up all of them
  const int lane = threadIdx.x & 31;
  uint32_t c[kFT / 32], sum = 0;
#pragma unroll
  for (int i = 0; i < kFT / 32; ++i) sum += c[i] = hist[lane * (kFT / 32) + i];
  uint32_t pre = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, pre, o);
    if (lane >= o) pre += x;
  }
  pre -= sum;
  uint32_t at = 0xffffffffu;
#pragma unroll
  for (int i = 0; i < kFT / 32; ++i) {
    if (pre < k && pre + c[i] >= k) at = lane * (kFT / 32) + i;
    pre += c[i];
  }
  at = __reduce_min_sync(0xffffffffu, at);
  cta_sync();
  hist[threadIdx.x] = 0;
  cta_sync();
  if (at != 0xffffffffu) return top - at;
  uint32_t t = 0;
  for (int bit = 15; bit >= 0; --bit) {
    const uint32_t trial = t | (1u << bit);
    if (cta_count(mine >= trial) >= (int)k) t = trial;
  }
  return t;
}

// Bin where the running sum of 256 bins, taken from `bin 0` on, reaches (kCount: of
// counts) `target`; sh.bin (kListBins: it does not) and the sum before it in sh.above.
template <bool kCount>
__device__ __forceinline__ void find_bin(FilterShared& sh, const FilterLists& ls, unsigned long long target) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    unsigned long long v[kListBins / 32], mine = 0;
#pragma unroll
    for (int i = 0; i < kListBins / 32; ++i) {
      const int bin = lane * (kListBins / 32) + i;
      v[i] = kCount ? ls.count[bin] : ls.mass[bin];
      mine += v[i];
    }
    unsigned long long pre = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long x = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += x;
    }
    if (lane == 0) sh.bin = kListBins, sh.in_bin = 0;
    __syncwarp();
    pre -= mine;
#pragma unroll
    for (int i = 0; i < kListBins / 32; ++i) {
      if (pre < target && pre + v[i] >= target) {
        sh.bin = lane * (kListBins / 32) + i;
        sh.above = pre;
      }
      pre += v[i];
    }
  }
  cta_sync();
}

// Where column i of a list lies: one after another, or each CTA's in its own part.
struct ListMap {
  int C;  // parts, or 0
  int slot;
  __device__ __forceinline__ int at(const FilterShared& sh, int i) const {
    if (!C) return i;
    int j = i, found = 0;
    for (int r = 0; r < C; ++r) {
      const int n = (int)sh.counts[slot][r];
      if (j >= 0 && j < n) found = r * (kListCap / C) + j;
      j -= n;
    }
    return found;
  }
};

// What a row's answer needs of its kept columns, in CTA 0.
// (A probability is of the weight itself: of one of next to nothing the list's units hold few bits.)
template <bool kVerify>
__device__ __forceinline__ void answer_draw(const FilterParams& p, const FilterShared& sh, const Scale& sc, int row,
                                            unsigned long long key, unsigned long long W) {
  const int col = (int)(0xffffffffu - (uint32_t)key);
  if (kVerify) {
    p.cuts[row].token = col;
  } else {
    p.out_tokens[row] = col;
    if (p.out_prob) p.out_prob[row] = ratio(weight(sc, sh.table, key_value(key_of(key))), W, kListBits);
  }
}
template <bool kVerify, int kPer>
__device__ __forceinline__ void keep_record(const FilterParams& p, FilterShared& sh, const Scale& sc, int row, float T, int draft,
                                            unsigned long long W, const bool (&keep)[kPer], const unsigned long long (&key)[kPer],
                                            const unsigned long long (&w)[kPer]) {
  const bool store = row < p.na;
#pragma unroll
  for (int h = 0; h < kPer; ++h) {
    if (keep[h]) {
      const int col = (int)(0xffffffffu - (uint32_t)key[h]);
      if (col == draft) {
        const float2 f = weight(sc, sh.table, key_value(key_of(key[h])));
        sh.wx = (double)f.x + (double)f.y;
      }
      if (store) {
        const uint32_t at = atomicAdd(&sh.stored, 1u);
        if (at < kKeptCap) {
          Kept& o = p.kept[(long long)row * kKeptCap + at];
          o.w = w[h];
          o.col = col;
        }
      }
    }
  }
  cta_sync();
  if (threadIdx.x == 0) {
    unsigned long long least = ~0ull;
    for (int x = 0; x < kFW; ++x) least = min(least, sh.warp_sum[x]);
    RowCut& c = p.cuts[row];
    c.cut.key = key_of(least);
    c.cut.tie = (int)(0xffffffffu - (uint32_t)least);
    c.cut.floor = -INFINITY;
    c.M = sc.M;
    c.T = T;
    c.listed = store && sh.stored <= kKeptCap ? (int)sh.stored : -1;
    c.W = (double)W * (1.0 / (1ull << kListBits));
    c.wx = sh.wx;  // (a token outside [0,V) is no listed column)
  }
}

// A short list, one column a thread: ranks, preceding weights and running sums in column
// order by comparing all pairs.  (Bins, as below, take fewer steps but more barriers.)
template <bool kVerify>
__device__ __forceinline__ void resolve_pairs(const FilterParams& p, FilterShared& sh, FilterLists& ls, const Scale& sc, int row,
                                              int L, ListMap map, int k, float share, unsigned long long whole, float floor, float T,
                                              float u, bool draws, int draft) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  ulonglong2* pair = reinterpret_cast<ulonglong2*>(&ls);
  unsigned long long key[1] = {0}, w[1] = {0};
  if (tid < L) key[0] = sh.list[map.at(sh, tid)];
  if (L > k + 8) {  // the CTAs' lists overlap: the first k of them, and a few more
    const uint32_t mine = tid < L ? key_of(key[0]) >> 16 : 0u;
    const uint32_t bound = kth_prefix(sh.hist, mine, value_key(sc.M) >> 16, (uint32_t)k);
    if (tid == 0) sh.own = 0;
    cta_sync();
    if (tid < L && mine >= bound) sh.list[atomicAdd(&sh.own, 1u)] = key[0];
    cta_sync();
    L = (int)sh.own;
    if (tid < L) key[0] = sh.list[tid];
  }
  bool keep[1] = {tid < L};
  const bool on = 32 * warp < L;  // this warp has columns
  if (on) {
    if (keep[0]) w[0] = fixed_weight(weight(sc, sh.table, key_value(key_of(key[0]))), kListBits);
    pair[tid] = make_ulonglong2(key[0], w[0]);
  }
  if (tid == 0) {
    sh.above = 0;
    if (kVerify) {
      sh.stored = 0;
      sh.wx = 0.0;
    }
  }
  cta_sync();
  int rank = 0;
  unsigned long long pre = 0;
  if (on) {
    unsigned long long pre2 = 0;
#pragma unroll 2
    for (int j = 0; j + 1 < L; j += 2) {
      const ulonglong2 o = pair[j], o2 = pair[j + 1];
      const bool first = o.x > key[0], first2 = o2.x > key[0];
      rank += first + first2;
      pre += first ? o.y : 0ull;
      pre2 += first2 ? o2.y : 0ull;
    }
    pre += pre2;
    if (L & 1) {
      const ulonglong2 o = pair[L - 1];
      rank += o.x > key[0];
      pre += o.x > key[0] ? o.y : 0ull;
    }
    if (keep[0] && rank == min(k, L) - 1) sh.total = pre + w[0];
  }
  cta_sync();
  if (on) {
    if (keep[0] && share < 1.f)
      keep[0] = whole ? (pre >> (kListBits - kSumBits)) < share_from(share, whole) : pre < share_from(share, sh.total);
    keep[0] = keep[0] && rank < k && key_value(key_of(key[0])) >= floor;
    if (!keep[0]) w[0] = 0;
    pair[tid].y = w[0];
    const unsigned long long sum = warp_sum_u64(w[0]);
    if (lane == 0) atomicAdd(&sh.above, sum);
  }
  if (kVerify) {
    unsigned long long least = keep[0] ? key[0] : ~0ull;
#pragma unroll
    for (int o = 16; o; o >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
    if (lane == 0) sh.warp_sum[warp] = least;
  }
  cta_sync();
  const unsigned long long W = sh.above;
  if (draws && keep[0] && w[0]) {
    const unsigned long long at = share_of(u, W);
    const uint32_t inv = (uint32_t)key[0];  // larger: a lower column
    unsigned long long upto = 0, upto2 = 0;
#pragma unroll 2
    for (int j = 0; j + 1 < L; j += 2) {
      const ulonglong2 o = pair[j], o2 = pair[j + 1];
      upto += (uint32_t)o.x >= inv ? o.y : 0ull;
      upto2 += (uint32_t)o2.x >= inv ? o2.y : 0ull;
    }
    upto += upto2;
    if ((L & 1) && (uint32_t)pair[L - 1].x >= inv) upto += pair[L - 1].y;
    if (upto > at && upto - w[0] <= at) answer_draw<kVerify>(p, sh, sc, row, key[0], W);
  }
  if (kVerify) keep_record<kVerify, 1>(p, sh, sc, row, T, draft, W, keep, key, w);
}

// CTA 0 of a row whose kept columns are all among the L listed ones: the cut and the draw
// in linear time, by bins of the value (from the largest on) and of the column, with all
// pairs compared within one bin only.  Weights are integers here (2^kListBits for the
// largest), sums exact.
//  k: columns kept at most; share: of the weight (from 1 on: all); whole: the row's weight
//  times 2^kSumBits, or 0: that of the first k.
//  kCutOnly: the listed columns follow others, of weight `above` (as whole) in all, that are kept; the last
//  kept column goes to every CTA's sh.cut_key and sh.cut_tie.
template <bool kVerify, bool kCutOnly>
__device__ __forceinline__ void resolve_list(const FilterParams& p, FilterShared& sh, FilterLists& ls, const Scale& sc, int row,
                                             int L, ListMap map, uint32_t low, uint32_t top, int k, float share, unsigned long long whole,
                                             float floor, float T, float u, bool draws, int draft, int C, unsigned long long above) {
  constexpr int kPer = kListCap / kFT;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned long long key[kPer], w[kPer];
  bool keep[kPer];
  uint32_t bin[kPer];
  const float per_bin = (float)kListBins / ((float)(top - low) + 1.f);
#pragma unroll
  for (int h = 0; h < kPer; ++h) {
    const int i = tid + h * kFT;
    keep[h] = i < L;
    key[h] = w[h] = bin[h] = 0;
    if (keep[h]) {
      key[h] = sh.list[map.at(sh, i)];
      w[h] = fixed_weight(weight(sc, sh.table, key_value(key_of(key[h]))), kListBits);
      bin[h] = min((uint32_t)((float)(top - key_of(key[h])) * per_bin), (uint32_t)kListBins - 1);
    }
  }
  auto clear = [&]() {
    if (tid < kListBins) ls.mass[tid] = 0, ls.count[tid] = 0;
    cta_sync();
  };
  auto select = [&](bool in, int h) {
    if (in) {
      const uint32_t at = atomicAdd(&sh.in_bin, 1u);
      ls.sel.key[at] = key[h];
      ls.sel.w[at] = w[h];
    }
  };

  if (L > k) {  // the first k
    clear();
#pragma unroll
    for (int h = 0; h < kPer; ++h)
      if (keep[h]) atomicAdd(&ls.count[bin[h]], 1u);
    cta_sync();
    find_bin<true>(sh, ls, (unsigned long long)k);
#pragma unroll
    for (int h = 0; h < kPer; ++h) select(keep[h] && bin[h] == sh.bin, h);
    cta_sync();
    const int n = (int)sh.in_bin;
#pragma unroll
    for (int h = 0; h < kPer; ++h) {
      if (keep[h] && bin[h] >= sh.bin) {
        uint32_t r = (uint32_t)sh.above;
        if (bin[h] == sh.bin)
          for (int j = 0; j < n; ++j) r += ls.sel.key[j] > key[h];
        keep[h] = bin[h] == sh.bin && r < (uint32_t)k;
      }
    }
    cta_sync();
  }
  if (share < 1.f) {  // the smallest prefix that holds its share
    clear();
#pragma unroll
    for (int h = 0; h < kPer; ++h)
      if (keep[h]) atomicAdd(&ls.mass[bin[h]], w[h]);
    cta_sync();
    if (whole == 0) {
      if (tid < 32) {
        unsigned long long v = 0;
#pragma unroll
        for (int i = 0; i < kListBins / 32; ++i) v += ls.mass[lane + 32 * i];
        v = warp_sum_u64(v);
        if (lane == 0) sh.total = v;
      }
      cta_sync();
    }
    // (a sum of 2^kListBits is below the target exactly when it is below the next whole number)
    unsigned long long target = share_from(share, whole ? whole : sh.total);
    if (kCutOnly) target = target > above ? target - above : 1ull;
    // (a flat row's share may be more than 2^64 in the list's units: more than any list holds, where min-p left
    // out what the share would have kept)
    if (whole) target = min(target, ~0ull >> (kListBits - kSumBits)) << (kListBits - kSumBits);
    find_bin<false>(sh, ls, target);
#pragma unroll
    for (int h = 0; h < kPer; ++h) select(keep[h] && bin[h] == sh.bin, h);
    cta_sync();
    const int n = (int)sh.in_bin;
#pragma unroll
    for (int h = 0; h < kPer; ++h) {
      if (keep[h] && bin[h] >= sh.bin) {
        unsigned long long before = sh.above;
        if (bin[h] == sh.bin)
          for (int j = 0; j < n; ++j)
            if (ls.sel.key[j] > key[h]) before += ls.sel.w[j];
        keep[h] = bin[h] == sh.bin && before < target;
      }
    }
    cta_sync();
  }

  unsigned long long least = ~0ull;
  if (kCutOnly) {
#pragma unroll
    for (int h = 0; h < kPer; ++h)
      if (keep[h]) least = min(least, key[h]);
#pragma unroll
    for (int o = 16; o; o >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
    if (lane == 0) sh.warp_sum[warp] = least;
    cta_sync();
    if (tid < C) {
      for (int x = 0; x < kFW; ++x) least = min(least, sh.warp_sum[x]);
      *at_rank(&sh.cut_key, tid) = key_of(least);
      *at_rank(&sh.cut_tie, tid) = (int)(0xffffffffu - (uint32_t)least);
    }
    return;
  }

  // what is kept, by bins of the column
  clear();
  const float per_col = (float)kListBins / (float)p.V;
#pragma unroll
  for (int h = 0; h < kPer; ++h) {
    keep[h] = keep[h] && key_value(key_of(key[h])) >= floor;
    if (keep[h]) {
      bin[h] = min((uint32_t)((float)(0xffffffffu - (uint32_t)key[h]) * per_col), (uint32_t)kListBins - 1);
      atomicAdd(&ls.mass[bin[h]], w[h]);
      least = min(least, key[h]);
    }
  }
  if (kVerify) {
#pragma unroll
    for (int o = 16; o; o >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
    if (lane == 0) sh.warp_sum[warp] = least;
    if (tid == 0) {
      sh.stored = 0;
      sh.wx = 0.0;
    }
  }
  cta_sync();
  if (tid < 32) {
    unsigned long long v = 0;
#pragma unroll
    for (int i = 0; i < kListBins / 32; ++i) v += ls.mass[lane + 32 * i];
    v = warp_sum_u64(v);
    if (lane == 0) sh.total = v;
  }
  cta_sync();
  const unsigned long long W = sh.total;
  if (draws) {
    const unsigned long long at = share_of(u, W);
    find_bin<false>(sh, ls, at + 1);
#pragma unroll
    for (int h = 0; h < kPer; ++h) select(keep[h] && bin[h] == sh.bin, h);
    cta_sync();
    const int n = (int)sh.in_bin;
#pragma unroll
    for (int h = 0; h < kPer; ++h) {
      if (keep[h] && w[h] && bin[h] == sh.bin) {
        const uint32_t inv = (uint32_t)key[h];  // larger: a lower column
        unsigned long long upto = sh.above;
        for (int j = 0; j < n; ++j)
          if ((uint32_t)ls.sel.key[j] >= inv) upto += ls.sel.w[j];
        if (upto > at && upto - w[h] <= at) answer_draw<kVerify>(p, sh, sc, row, key[h], W);
      }
    }
  }
  if (kVerify) keep_record<kVerify, kPer>(p, sh, sc, row, T, draft, W, keep, key, w);
}

template <int DT, bool kVerify>
__global__ void __launch_bounds__(kFT, 4) filter_kernel(const FilterParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  FilterShared& sh = *reinterpret_cast<FilterShared*>(smem);
  unsigned char* room = smem + ((sizeof(FilterShared) + 127) & ~(size_t)127);
  FilterLists& ls = *reinterpret_cast<FilterLists*>(room);
  uint4* data = reinterpret_cast<uint4*>(room);
  using E = Elt<DT>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster_rank();
  const int row = blockIdx.x / p.C;

  // ---- which row
  const char* src;
  int ask, draft = 0;
  bool draws = true, ok = true;
  if (kVerify) {
    if (row < p.na) {
      ask = row / (p.Kp + 1);
      draws = row - ask * (p.Kp + 1) == p.Kp;
      src = p.rows_a + (long long)row * p.a_bytes;
    } else {
      const int r = row - p.na;
      ask = r / p.Kp;
      draws = false;
      src = p.rows_b + (long long)r * p.b_bytes;
    }
  } else {
    ask = row / p.per;
    const int i = p.sample_idx ? __ldg(p.sample_idx + row) : row;
    ok = i >= 0 && i < p.src_rows;
    src = p.rows_a + (long long)(ok ? i : 0) * p.a_bytes;
  }

  // ---- its slice is on the way before anything else is looked at
  Slice<DT> s;
  s.v = data;
  s.lane = lane;
  s.warp = warp;
  s.rank = rank;
  s.C = p.C;
  s.sh = &sh;
  s.turn = 0;
  const int v0 = rank * p.per_cta;
  s.n = max(0, min(p.per_cta, p.nvec - v0));
  s.lo = min(s.n, warp * p.seg);
  s.hi = min(s.n, s.lo + p.seg);
  s.col0 = v0 * E::kN;
  uint32_t phase = 0;
  auto start_load = [&]() {
    if (lane == 0) {
      const int whole = min(s.hi, p.V / E::kN - v0);  // vectors that lie in the row as a whole
      const int bytes = max(0, whole - s.lo) * 16;
      mbar_arrive_expect_tx(&sh.bars[warp], bytes);
      if (bytes) bulk_load(data + s.lo, src + (long long)(v0 + s.lo) * 16, bytes, &sh.bars[warp]);
    }
  };
  const int part = p.V % E::kN;
  auto finish_load = [&]() {
    // the row's last columns, where they do not fill a vector
    if (part && s.hi > s.lo && v0 + s.hi == p.nvec && lane < E::kN) {
      const int col = (p.nvec - 1) * E::kN + lane;
      const float x = lane < part ? E::load(src, col) : -INFINITY;
      if (DT == PE_BF16)
        reinterpret_cast<unsigned short*>(data + s.hi - 1)[lane] = (unsigned short)(__float_as_uint(x) >> 16);
      else
        reinterpret_cast<float*>(data + s.hi - 1)[lane] = x;
    }
    if (!mbar_wait(&sh.bars[warp], phase)) {
      if (lane == 0) atomicOr(p.err, PE_ERR_TIMEOUT);
      (void)mbar_wait(&sh.bars[warp], phase);
    }
    phase ^= 1u;
    __syncwarp();
  };
  if (lane == 0) {
    mbar_init(&sh.bars[warp], 1);
    mbar_init_fence();
  }
  start_load();

  // ---- which parameters (the same in every CTA of the cluster)
  if (!ok && rank == 0 && tid == 0) atomicOr(p.err, PE_ERR_ROW_RANGE);
  if (kVerify) {
    if (row >= p.na) draft = __ldg(p.tokens + ask * (p.Kp + 1) + (row - p.na - ask * p.Kp) + 1);
    else if (!draws) draft = __ldg(p.tokens + row + 1);
  }
  Asked a;
  if (!read_asked(p.asked, ask, p.V, a)) {
    ok = false;
    if (rank == 0 && tid == 0) atomicOr(p.err, PE_ERR_PARAM);
  }
  float u = 0.f;
  if (draws) {
    u = __ldg(p.u + (kVerify ? ask : row));
    if (!(u >= 0.f && u < 1.f)) {
      ok = false;
      if (rank == 0 && tid == 0) atomicOr(p.err, PE_ERR_PARAM);
    }
  }
  // what a row without an answer gets
  auto none = [&](double W) {
    if (rank != 0 || tid != 0) return;
    if (kVerify) {
      // (all of it: the residual pass chooses its arithmetic by the cuts of both rows)
      RowCut& c = p.cuts[row];
      c.cut.key = 0;
      c.cut.tie = INT32_MAX;
      c.cut.floor = -INFINITY;
      c.M = 0.f;
      c.T = a.T;
      c.listed = 0;
      c.token = -1;
      c.W = W;
      c.wx = 0.0;
    } else {
      p.out_tokens[row] = -1;
      if (p.out_prob) p.out_prob[row] = 0.f;
    }
  };
  if (tid == 0) {
    sh.own = 0;
  }
  if (tid < 32) sh.table[tid] = kExp2Table[tid];
  sh.hist[tid] = 0;
  if (tid == 32) sh.rates = make_rates(a.T, a.m);
  __syncwarp();
  cluster_arrive();
  finish_load();
  if (!ok) {  // (not before its copies have landed)
    cluster_wait();
    none(-1.0);
    return;
  }

  // ---- maxima
  float tmax = -INFINITY;
#pragma unroll 4
  for (int i = s.lo + lane; i < s.hi; i += 32) tmax = fmaxf(tmax, E::max_of(s.v[i]));
  const uint32_t mine = ordered_bits(tmax);
  const uint32_t wmax = __reduce_max_sync(0xffffffffu, mine);
  if (lane == 0) sh.warp_count[warp] = wmax;
  cta_sync();
  uint32_t top = 0;
#pragma unroll
  for (int w = 0; w < kFW; ++w) top = max(top, sh.warp_count[w]);
  const bool small_k = a.k <= kListK && a.k < p.V;
  const bool nucleus = a.k == p.V && a.p < 1.f;
  // every CTA's own first k columns, where that makes a short list
  bool local = small_k && a.k * p.C <= kListCap / 2;
  uint32_t bound = 0, fair = 0;
  if (small_k) {
    bound = a.k == 1 ? top >> 16 : kth_prefix(sh.hist, mine >> 16, top >> 16, (uint32_t)a.k);
    if (!local) fair = kth_prefix(sh.hist, mine >> 16, top >> 16, (uint32_t)(a.k + p.C - 1) / p.C);
  }
  const float p_mass = a.p > 0.f ? a.p : 0.f;
  unsigned long long Z = 0;  // the whole row's weight (top-p alone)
  unsigned long long large[2] = {0, 0};
  cluster_wait();  // every CTA has started
  if (!local) {
    if (tid < p.C) {
      *at_rank(&sh.maxima[rank], tid) = top;
      if (small_k) {
        *at_rank(&sh.bounds[rank], tid) = bound;
        *at_rank(&sh.shares[rank], tid) = fair;
      }
    }
    cluster_sync();
    for (int r = 0; r < p.C; ++r) top = max(top, sh.maxima[r]);
    if (small_k) {
      // k columns lie from the largest of the bounds on, and from the smallest of the CTAs' shares on
      for (int r = 0; r < p.C; ++r) {
        bound = max(bound, sh.bounds[r]);
        fair = min(fair, sh.shares[r]);
      }
      bound = max(bound, fair);
    }
  }
  float M = key_value(top);  // local: of this CTA's columns only
  auto empty = [&]() {
    if (rank == 0 && tid == 0) atomicOr(p.err, PE_ERR_EMPTY_ROW);
    none(0.0);
  };
  if (!local && M == -INFINITY) return empty();

  // the floor of min-p, once M is the row's
  auto floor_of = [&]() -> float {
    if (!(a.m > 0.f)) return -INFINITY;
    if (tid == 0) sh.floor = min_p_floor(a, sh.rates, M);
    cta_sync();
    return sh.floor;
  };
  float floor = local ? -INFINITY : floor_of();
  Scale sc = make_scale(M, sh.rates);

  Cut cut;
  cut.key = 0;
  cut.tie = INT32_MAX;
  cut.floor = -INFINITY;  // (min-p comes last: the others' shares are of columns below its floor too)

  // Gather the columns with keys in [low, high] that the cut so far keeps into CTA 0's list;
  // their number, and where they lie.
  const int part_cap = kListCap / p.C;
  auto gather = [&](uint32_t low, uint32_t high, ListMap& map) -> int {
    unsigned long long* list = at_rank(sh.list, 0);
    const float low_x = key_value(max(low, 0x007fffffu));  // (below the key of -infinity lie NaNs)
    // Vectors that hold any go to a queue of the warp; then its lanes take an element each (a
    // lane with its whole vector, as it comes, takes four times as long: the others wait).
    auto scan = [&](uint32_t first, uint32_t most) {
      if (!__any_sync(0xffffffffu, tmax >= low_x)) return;
      uint32_t queued = 0;
      auto take = [&](uint32_t n) {
        __syncwarp();
        for (uint32_t j0 = 0; j0 < n; j0 += 32 / E::kN) {
          const uint32_t j = j0 + lane / E::kN;
          uint32_t k = 0;
          int col = 0;
          bool in = j < n;
          if (in) {
            const int i = sh.hits[warp][j], e = lane % E::kN;
            const float x = E::element(s.v, i, e);
            k = ordered_bits(x);
            col = s.col0 + i * E::kN + e;
            in = x >= low_x && k <= high && col < p.V && (k != cut.key || col <= cut.tie);
          }
          const uint32_t m = __ballot_sync(0xffffffffu, in);
          if (m) {
            uint32_t at = 0;
            if (lane == 0) at = atomicAdd(&sh.own, (uint32_t)__popc(m));
            at = __shfl_sync(0xffffffffu, at, 0) + __popc(m & ((1u << lane) - 1));
            if (in && at < most) list[first + at] = ((unsigned long long)k << 32) | (0xffffffffu - (uint32_t)col);
          }
        }
        __syncwarp();
      };
#pragma unroll 2
      for (int i0 = s.lo; i0 < s.hi; i0 += 32) {
        const int i = i0 + lane;
        const bool hit = i < s.hi && E::max_of(s.v[i]) >= low_x;
        const uint32_t m = __ballot_sync(0xffffffffu, hit);
        if (!m) continue;
        if (hit) sh.hits[warp][queued + __popc(m & ((1u << lane) - 1))] = (unsigned short)i;
        queued += __popc(m);
        if (queued > 32) {  // (room for another 32 is needed)
          take(queued);
          queued = 0;
        }
      }
      take(queued);
    };
    scan((uint32_t)(rank * part_cap), (uint32_t)part_cap);  // each CTA in its part of the list
    cta_sync();
    map.C = p.C;
    map.slot = s.turn & 1;
    if (tid < p.C) {
      *at_rank(&sh.counts[map.slot][rank], tid) = sh.own;
      if (local) *at_rank(&sh.maxima[rank], tid) = top;
    }
    cluster_sync();
    ++s.turn;
    uint32_t L = 0, before = 0, most = 0;
    for (int r = 0; r < p.C; ++r) {
      const uint32_t n = sh.counts[map.slot][r];
      if (r == rank) before = L;
      L += n;
      most = max(most, n);
    }
    if (most > (uint32_t)part_cap && L <= kListCap) {  // some part is too short: one after another
      if (tid == 0) sh.own = 0;
      cta_sync();
      scan(before, kListCap);
      cluster_sync();
      map.C = 0;
    }
    return (int)L;  // (at most 2^18)
  };

  // ---- rows whose kept columns all reach a known value: a list
  float octaves = 0.f;  // how far below M the cut lies at most
  const bool by_min = a.k == p.V && a.p >= 1.f && floor > -INFINITY;
  if (small_k || nucleus || by_min) {
    uint32_t low = small_k ? bound << 16 : value_key(floor);
    if (nucleus) {
      Z = s.mass(sc, large);
      if (lane == 0) {
        sh.warp_sum[warp] = Z;
        sh.warp_large[0][warp] = large[0];
        sh.warp_large[1][warp] = large[1];
      }
      cta_sync();
      if (tid < 3 * p.C) {
        const unsigned long long* part = tid < p.C ? sh.warp_sum : sh.warp_large[tid / p.C - 1];
        unsigned long long sum = 0;
        for (int w = 0; w < kFW; ++w) sum += part[w];
        *at_rank(tid < p.C ? &sh.sums[0][rank] : &sh.large[tid / p.C - 1][rank], tid % p.C) = sum;
      }
      cluster_sync();
      Z = large[0] = large[1] = 0;
      for (int r = 0; r < p.C; ++r) {
        Z += sh.sums[0][r];
        large[0] += sh.large[0][r];
        large[1] += sh.large[1][r];
      }
      // The last kept column and those after it weigh more than (1 - p) Z and are at most
      // V, so it weighs more than (1 - p) Z / V (and a little less, for this estimate's roundings).
      octaves = 0x1p-16f - log2f((1.f - p_mass) * ((float)Z * 0x1p-44f) / (float)p.V);
      float away = octaves;
      // Where what is large holds the share by itself, that is the list.
      const float need = (p_mass + 0x1p-16f) * (float)Z;
      if ((float)large[0] > need) away = fminf(away, 8.f);
      else if ((float)large[1] > need) away = fminf(away, 12.f);
      away *= sc.octave;
      low = max(low, M == INFINITY ? top : value_key(M - away - 0x1p-20f * (fabsf(M) + away)));
    }
    ListMap map;
    const int L = gather(low, 0xffffffffu, map);
    if (local) {
      for (int r = 0; r < p.C; ++r) top = max(top, sh.maxima[r]);
      M = key_value(top);
      if (M == -INFINITY) return empty();
      sc = make_scale(M, sh.rates);
    }
    if (L <= kListCap) {
      if (rank == 0) {
        if (local) floor = floor_of();
        const int k = small_k ? a.k : p.V;
        const float share = a.p < 1.f ? p_mass : 1.f;
        const unsigned long long whole = nucleus ? Z : 0ull;
        if (L <= kPairs)
          resolve_pairs<kVerify>(p, sh, ls, sc, row, L, map, k, share, whole, floor, a.T, u, draws, draft);
        else
          resolve_list<kVerify, false>(p, sh, ls, sc, row, L, map, low, top, k, share, whole, floor, a.T, u, draws, draft, p.C, 0ull);
      }
      return;
    }
    if (local) floor = floor_of();
    local = false;
  }

  // ---- the cut, over the whole row: a histogram shows between which values it lies, what is
  // above is added up, and a list of the columns between them decides
  auto refine = [&](bool by_count, float range, double target, int k, unsigned long long whole) -> bool {
    if (M == INFINITY) return false;
    float lo_x, hi_x;
    const bool found = by_count ? s.template steer<false>(sc, cut, range, target, sh.steps, lo_x, hi_x)
                                : s.template steer<true>(sc, cut, range, target, sh.steps, lo_x, hi_x);
    if (!found) return false;
    if (tid == 0) sh.own = 0;
    uint32_t n = 0;
    unsigned long long sum = 0;
    const uint32_t high = hi_x == INFINITY ? 0xffffffffu : value_key(hi_x);
    if (high != 0xffffffffu) {  // (what the cut so far leaves out is below)
      if (by_count) s.template above<false>(sc, high, n, sum);
      else s.template above<true>(sc, high, n, sum);
    } else {
      cluster_sync();
    }
    const uint32_t low = value_key(lo_x);
    ListMap map;
    const int L = gather(low, high - 1, map);
    if (L == 0 || L > kListCap) return false;
    if (rank == 0)
      resolve_list<kVerify, true>(p, sh, ls, sc, row, L, map, low, min(high - 1, top), by_count ? k - (int)n : p.V,
                                  by_count ? 1.f : p_mass, whole, floor, a.T, u, draws, draft, p.C, sum);
    cluster_sync();
    if (rank == 0) {  // its slice again: the list's bins took its place
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      cta_sync();
      start_load();
      finish_load();
    }
    cut.key = sh.cut_key;
    cut.tie = sh.cut_tie;
    return true;
  };
  if (a.k < p.V && !refine(true, 63.f, (double)a.k, a.k, 0ull)) {
    cut.key = s.template search<false>(sc, (uint32_t)a.k, 0.0);
    uint32_t c = 0;
    unsigned long long sum;
    if (cut.key != 0xffffffffu) s.template above<false>(sc, cut.key + 1, c, sum);
    cut.tie = s.nth_tie(cut.key, (uint32_t)a.k - c);
  }
  if (a.p < 1.f) {
    uint32_t c = 0;
    unsigned long long sum = Z;
    if (a.k < p.V) {
      sum = s.kept_mass(sc, cut);
      s.exchange(c, sum);
      octaves = 0x1p-16f - log2f((1.f - p_mass) * ((float)sum * 0x1p-44f) / (float)a.k);
    }
    const double whole = (double)sum;
    if (!refine(false, fminf(octaves + 0x1p-8f, 63.f), fmax((double)p_mass * whole * 0x1p-44, 0x1p-40), 0, sum)) {
      const uint32_t key_k = cut.key;
      const int tie_k = cut.tie;
      const double target = (double)p_mass * whole;
      uint32_t key_p = s.template search<true>(sc, 0u, target);
      if (target <= 0.0) key_p = top;  // the first column alone
      if (key_p < key_k) key_p = key_k;
      s.template above<true>(sc, key_p + 1, c, sum);
      const float2 w = weight(sc, sh.table, key_value(key_p));
      const double one = ((double)w.x + (double)w.y) * (double)(1ull << kSumBits);
      double need = ceil((target - (double)sum) / one);
      if (!(need >= 1.0)) need = 1.0;
      cut.key = key_p;
      cut.tie = s.nth_tie(key_p, need < 4e9 ? (uint32_t)need : 0xffffffffu);
      if (key_p == key_k) cut.tie = min(cut.tie, tie_k);
    }
  }


  // ---- the kept weight, and the draw
  cut.floor = floor;
  uint32_t c = 0;
  unsigned long long sum, before = 0;
  uint32_t c_before = 0;
  auto kept = [&](int i, int from, int to, WeightSum<256>& ws) {
    const uint4 q = s.v[i];
#pragma unroll
    for (int e = 0; e < E::kN; ++e) {
      const float x = E::get(q, e);
      if (e >= from && e < to && cut.keeps(x, s.col0 + i * E::kN + e)) {
        const float2 w = weight(sc, sh.table, x);
        ws.add(w.x, w.y);
      }
    }
  };
  unsigned long long mine_w;
  if (cut.key == 0 && floor == -INFINITY) {  // every column
    mine_w = s.mass(sc, large);
  } else {
    mine_w = s.kept_mass(sc, cut);
  }
  sum = mine_w;
  s.exchange(c, sum, &before, &c_before);
  if (kVerify && rank == 0 && tid == 0) {
    RowCut& o = p.cuts[row];
    o.cut = cut;
    o.M = M;
    o.T = a.T;
    o.listed = -1;
    o.W = (double)sum * (1.0 / (1ull << kSumBits));
    double wx = 0.0;
    if (draft >= 0 && draft < p.V) {
      const float x = E::load(src, draft);
      if (cut.keeps(x, draft)) {
        const float2 w = weight(sc, sh.table, x);
        wx = (double)w.x + (double)w.y;
      }
    }
    o.wx = wx;
  }
  if (draws) {
    const unsigned long long at = share_of(u, sum);
    unsigned long long pre;
    const int chosen = narrow<DT>(s, sh, p.seg, 0, s.n, at, before, pre, [&]() { return s.kept_mass(sc, cut); });
    if (warp == chosen) {
      const int i = find_column<E::kN, 256>(s.lo, s.hi, lane, at > pre ? at - pre : 0ull, kSumBits, kept);
      if (lane == 0) {
        const int col = i < 0 ? -1 : s.col0 + i;
        if (i < 0) atomicOr(p.err, PE_ERR_INTERNAL);  // (a share that is not zero has a column of some weight)
        if (kVerify) {
          p.cuts[row].token = col;
        } else if (i < 0) {
          p.out_tokens[row] = -1;
          if (p.out_prob) p.out_prob[row] = 0.f;
        } else {
          p.out_tokens[row] = col;
          if (p.out_prob) p.out_prob[row] = ratio(weight(sc, sh.table, E::load(src, col)), sum, kSumBits);
        }
      }
    }
  }
}

}  // namespace pe

namespace pe {

// --------------------------------------------------------- the bonus token
template <int DT>
__device__ __forceinline__ uint4 row_vector(const char* row, int i, int V) {
  using E = Elt<DT>;
  if ((i + 1) * E::kN <= V) return __ldg(reinterpret_cast<const uint4*>(row) + i);
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (DT == PE_BF16) {
      const int col = i * 8 + 2 * j;
      const float lo = col < V ? E::load(row, col) : -INFINITY;
      const float hi = col + 1 < V ? E::load(row, col + 1) : -INFINITY;
      w[j] = (__float_as_uint(lo) >> 16) | (__float_as_uint(hi) & 0xffff0000u);
    } else {
      const int col = i * 4 + j;
      w[j] = __float_as_uint(col < V ? E::load(row, col) : -INFINITY);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Request b: the first rejected draft, then a draw from max(0, p - q) of its rows
// (from p where that is zero everywhere), or the bonus row's own draw.  p's kept
// columns come from the row's list where it has one: p - q is at most 0 elsewhere.
// Else both rows are read again, each warp its segment.
template <int DT>
__global__ void __launch_bounds__(kFT, 4) residual_kernel(const FilterParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  FilterShared& sh = *reinterpret_cast<FilterShared*>(smem);
  using E = Elt<DT>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster_rank();
  const int b = blockIdx.x / p.C;
  if (tid < 32) sh.table[tid] = kExp2Table[tid];
  if (tid == 0) sh.total = 0;
  cta_sync();
  cluster_arrive();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const RowCut* target = p.cuts + (long long)b * (p.Kp + 1);
  const RowCut* drafts = p.cuts + p.na + (long long)b * p.Kp;
  const bool bad = target[p.Kp].W < 0.0;
  if (warp == 0) {
    int a = p.Kp;
    for (int j0 = 0; j0 < p.Kp; j0 += 32) {
      const int j = j0 + lane;
      bool no = false;
      if (j < p.Kp) {
        const double pw = target[j].W, qw = drafts[j].W;
        // (a token outside [0,V): 0 and 0, rejected under any coin)
        const double px = pw > 0.0 ? target[j].wx / pw : 0.0, qx = qw > 0.0 ? drafts[j].wx / qw : 0.0;
        no = !((double)__ldg(p.coins + b * p.Kp + j) * qx < px);
        if (p.chance && rank == 0) p.chance[b * p.Kp + j] = bad || !(px > 0.0) ? 0.f : px < qx ? (float)(px / qx) : 1.f;
      }
      const uint32_t m = __ballot_sync(0xffffffffu, no);
      if (m && a == p.Kp) a = j0 + __ffs(m) - 1;
    }
    if (lane == 0) {
      sh.first = a;
      const RowCut& t = target[a];
      if (rank == 0) {
        p.accepted[b] = bad ? 0 : a;
        if (bad || t.W == 0.0) p.bonus[b] = -1;
        else if (a == p.Kp) p.bonus[b] = t.token;
      }
      if (!bad && a < p.Kp && t.W > 0.0) sh.rates = make_rates(t.T, 0.f);
    }
  }
  cta_sync();
  const int a = sh.first;
  const RowCut& t = target[a];
  const bool stream = t.listed < 0;
  cluster_wait();
  if (bad || a == p.Kp || t.W == 0.0) return;
  const RowCut& d = drafts[a];
  const char* trow = p.rows_a + ((long long)b * (p.Kp + 1) + a) * p.a_bytes;
  const char* drow = p.rows_b + ((long long)b * p.Kp + a) * p.b_bytes;
  const float u = __ldg(p.u + b);
  const bool has_q = d.W > 0.0;
  const Scale st = make_scale(t.M, sh.rates);
  const Scale sd = make_scale(has_q ? d.M : 0.f, sh.rates);
  const Cut ct = t.cut, cd = d.cut;
  constexpr int kBits = 60;

  if (!stream) {
    if (rank != 0) return;
    unsigned long long* w = reinterpret_cast<unsigned long long*>(smem + ((sizeof(FilterShared) + 127) & ~(size_t)127));
    int* cols = reinterpret_cast<int*>(w + kKeptCap);
    const Kept* kept = p.kept + ((long long)b * (p.Kp + 1) + a) * kKeptCap;
    const int L = min(t.listed, kKeptCap);
    unsigned long long mine = 0, whole = 0;
    int col = -1;
    if (tid < L) {
      col = kept[tid].col;
      const double pr = (double)kept[tid].w * (1.0 / (1ull << kListBits)) / t.W;
      double q = 0.0;
      if (has_q) {
        const float x = E::load(drow, col);
        if (cd.keeps(x, col)) {
          // (rounded as the list's weights are: rows alike have to leave exactly nothing)
          q = (double)fixed_weight(weight(sd, sh.table, x), kListBits) * (1.0 / (1ull << kListBits)) / d.W;
        }
      }
      whole = (unsigned long long)(pr * (double)(1ull << kBits) + 0.5);
      mine = pr > q ? (unsigned long long)((pr - q) * (double)(1ull << kBits) + 0.5) : 0ull;
    }
    const unsigned long long part = warp_sum_u64(mine);
    if (lane == 0 && part) atomicAdd(&sh.total, part);
    cta_sync();
    unsigned long long R = sh.total;
    cta_sync();
    if (R == 0) {
      mine = whole;
      const unsigned long long all = warp_sum_u64(mine);
      if (lane == 0 && all) atomicAdd(&sh.total, all);
      cta_sync();
      R = sh.total;
    }
    if (tid < kKeptCap) {
      w[tid] = mine;
      cols[tid] = tid < L ? col : INT32_MAX;
    }
    cta_sync();
    const unsigned long long at = share_of(u, R);
    if (mine) {
      unsigned long long upto = 0;
      for (int j = 0; j < L; ++j)
        if (cols[j] <= col) upto += w[j];
      if (upto > at && upto - mine <= at) p.bonus[b] = col;
    }
    return;
  }

  Slice<DT> s;
  s.lane = lane;
  s.warp = warp;
  s.rank = rank;
  s.C = p.C;
  s.sh = &sh;
  s.turn = 0;
  const int v0 = rank * p.per_cta, vn = max(0, min(p.per_cta, p.nvec - v0));
  s.lo = v0 + min(vn, warp * p.seg);
  s.hi = v0 + min(vn, warp * p.seg + p.seg);
  if (tid < 2) {  // 1 / W of both rows, as two floats
    const double i = tid == 0 ? 1.0 / t.W : has_q ? 1.0 / d.W : 0.0;
    const float hi = (float)i;
    sh.inverse[tid] = make_float2(hi, (float)(i - (double)hi));
  }
  cta_sync();
  const float ith = sh.inverse[0].x, itl = sh.inverse[0].y;
  const float idh = sh.inverse[1].x, idl = sh.inverse[1].y;
  bool with_q = has_q;
  // max(0, p - q) of one column, as the sum of two floats
  auto add_rest = [&](float xe, float ye, int col, WeightSum<2>& ws) {
    if (!ct.keeps(xe, col)) return;
    float2 w = weight(st, sh.table, xe);
    float ph = w.x * ith;
    float pl = fmaf(w.x, ith, -ph) + fmaf(w.x, itl, w.y * ith);
    if (with_q && cd.keeps(ye, col)) {
      w = weight(sd, sh.table, ye);
      const float qh = w.x * idh;
      const float ql = fmaf(w.x, idh, -qh) + fmaf(w.x, idl, w.y * idh);
      const float dh = ph - qh, bb = dh - ph;
      pl = ((ph - (dh - bb)) - (qh + bb)) + (pl - ql);
      ph = dh;
    }
    if (ph + pl > 0.f) ws.add(ph, pl);
  };
  auto rest = [&](int i, int from, int to, WeightSum<2>& ws) {
    for (int e = from; e < to; ++e) {
      const int col = i * E::kN + e;
      if (col < p.V) add_rest(E::load(trow, col), E::load(drow, col), col, ws);
    }
  };
  // the same of two small weights
  auto small_rest = [&](float xe, float ye) -> float {
    const float wt = small_weight<DT>(st, xe), wd = with_q ? small_weight<DT>(sd, ye) : 0.f;
    return fmaxf(fmaf(wt, itl, wt * ith) - fmaf(wd, idl, wd * idh), 0.f);
  };
  // The warp's share.  Vectors of small weights in both rows are added up as they come (as in
  // Slice::mass), where no cut asks for more; vectors below the
  // target's cut have nothing; the others are queued and taken an element a lane.
  const bool open = ct.key == 0 && ct.floor == -INFINITY && cd.key == 0 && cd.floor == -INFINITY && !st.inf && !(has_q && sd.inf);
  const float big_t = open ? st.M - 16.f * st.octave : fmaxf(key_value(max(ct.key, 0x007fffffu)), ct.floor);
  const float big_d = open && has_q ? sd.M - 16.f * sd.octave : INFINITY;
  auto share = [&]() -> unsigned long long {
    WeightSum<2> ws;
    uint32_t queued = 0;
    auto take = [&]() {
      __syncwarp();
      for (uint32_t j0 = 0; j0 < queued; j0 += 32 / E::kN) {
        const uint32_t j = j0 + lane / E::kN;
        if (j < queued) {
          const int e = lane % E::kN;
          rest(sh.hits[warp][j], e, e + 1, ws);
        }
      }
      queued = 0;
      __syncwarp();
    };
    uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
    if (s.lo + lane < s.hi) {
      x = row_vector<DT>(trow, s.lo + lane, p.V);
      y = row_vector<DT>(drow, s.lo + lane, p.V);
    }
    for (int i0 = s.lo; i0 < s.hi; i0 += 32) {
      const int i = i0 + lane;
      const uint4 cx = x, cy = y;
      if (i + 32 < s.hi) {  // the next ones ahead
        x = row_vector<DT>(trow, i + 32, p.V);
        y = row_vector<DT>(drow, i + 32, p.V);
      }
      bool put = false;
      if (i < s.hi) {
        put = E::max_of(cx) >= big_t || E::max_of(cy) >= big_d;
        if (!put && open) {
          float small = 0.f;
#pragma unroll
          for (int e = 0; e < E::kN; ++e) small += small_rest(E::get(cx, e), E::get(cy, e));
          ws.add(small, kSmallMean * small);
        }
      }
      const uint32_t m = __ballot_sync(0xffffffffu, put);
      if (m) {
        if (put) sh.hits[warp][queued + __popc(m & ((1u << lane) - 1))] = (unsigned short)i;
        queued += __popc(m);
        if (queued > 32) take();  // (room for another 32 is needed)
      }
    }
    take();
    return warp_sum_u64(ws.fixed(kBits));
  };
  unsigned long long sum = 0, before = 0;
  for (int turn = 0; turn < 2; ++turn) {
    sum = share();
    uint32_t c = 0, c_before = 0;
    s.exchange(c, sum, &before, &c_before);
    if (sum != 0) break;
    with_q = false;
  }
  auto no_column = [&]() {
    atomicOr(p.err, PE_ERR_INTERNAL);
    p.bonus[b] = -1;
  };
  if (sum == 0) {  // (p's weights are not all zero)
    if (rank == 0 && tid == 0) no_column();
    return;
  }
  // Vector by vector in the share's arithmetic: where p and q nearly agree, the other one may find
  // no column above zero in a share that is.
  auto alike = [&](int i, int from, int to, WeightSum<2>& ws) {
    if (open) {
      const uint4 x = row_vector<DT>(trow, i, p.V), y = row_vector<DT>(drow, i, p.V);
      if (!(E::max_of(x) >= big_t || E::max_of(y) >= big_d)) {
#pragma unroll
        for (int e = 0; e < E::kN; ++e)
          if (e >= from && e < to) {
            const float w = small_rest(E::get(x, e), E::get(y, e));
            ws.add(w, kSmallMean * w);
          }
        return;
      }
    }
    rest(i, from, to, ws);
  };
  const unsigned long long at = share_of(u, sum);
  unsigned long long pre;
  const int chosen = narrow<DT>(s, sh, p.seg, v0, v0 + vn, at, before, pre, [&]() {
    WeightSum<2> ws;
    for (int i = s.lo + lane; i < s.hi; i += 32) alike(i, 0, E::kN, ws);
    return warp_sum_u64(ws.fixed(kBits));
  });
  if (warp == chosen) {
    const int col = find_column<E::kN, 2>(s.lo, s.hi, lane, at > pre ? at - pre : 0ull, kBits, alike);
    if (lane == 0) {
      if (col >= 0) p.bonus[b] = col;
      else no_column();
    }
  }
}

}  // namespace pe

// ---------------------------------------------------------------- host side
namespace {

constexpr size_t kHeader = ((sizeof(pe::FilterShared) + 127) & ~(size_t)127);
constexpr int kMaxSmem = (int)kHeader + 64 * 1024;
constexpr int kRoomySlice = 52 * 1024;  // three CTAs and more on an SM

struct FilteredLayout {
  size_t kept_off, bytes;
  FilteredLayout(long long B, long long Kp) {
    const long long rows = B * (2 * Kp + 1);
    kept_off = (sizeof(pe::RowCut) * rows + 255) / 256 * 256;
    bytes = kept_off + sizeof(pe::Kept) * pe::kKeptCap * B * (Kp + 1);
  }
};

// CTAs of a row: as few as leave room for two CTAs on an SM, more while the rows
// do not fill the GPU.
void split_rows(pe::FilterParams& p, int elt, int sms) {
  const int epv = 16 / elt;
  p.nvec = (p.V + epv - 1) / epv;
  p.C = 1;
  while (p.C < pe::kMaxCluster &&
         (p.nvec * 16 / p.C > kRoomySlice || ((long long)p.n * p.C * 2 <= sms && p.C < 8 && p.nvec / p.C > 512)))
    p.C *= 2;
  p.per_cta = (p.nvec + p.C - 1) / p.C;
  p.seg = (p.per_cta + pe::kFW - 1) / pe::kFW;
}

template <int DT, bool kVerify>
int launch_filter(const pe::FilterParams& p, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  auto kernel = pe::filter_kernel<DT, kVerify>;
  static std::atomic<unsigned long long> wide{0};
  if (p.C > 8 && !pe_host::allow_wide_clusters(kernel, wide)) return PE_ECUDA;
  if (!pe_host::allow_smem(kernel, kMaxSmem, done)) return PE_ECUDA;
  const size_t slice = (size_t)p.per_cta * 16;
  const size_t smem = kHeader + (slice > sizeof(pe::FilterLists) ? slice : sizeof(pe::FilterLists));
  return pe_host::launch_clusters(pe::filter_kernel<DT, kVerify>, p.n * p.C, pe::kFT, p.C, smem, false, st, p) == cudaSuccess ? PE_OK : PE_ECUDA;
}

template <int DT>
int launch_verify(pe::FilterParams p, int B, int elt, int sms, cudaStream_t st) {
  const int rc = launch_filter<DT, true>(p, st);
  if (rc != PE_OK) return rc;
  p.n = B;
  split_rows(p, elt, sms);
  if (p.C > 8) {
    p.C = 8;
    p.per_cta = (p.nvec + 7) / 8;
    p.seg = (p.per_cta + pe::kFW - 1) / pe::kFW;
  }
  const size_t smem = kHeader + 12 * pe::kKeptCap;
  return pe_host::launch_clusters(pe::residual_kernel<DT>, B * p.C, pe::kFT, p.C, smem, true, st, p) == cudaSuccess ? PE_OK : PE_ECUDA;
}

int rows_ok(const void* rows, int64_t stride, int elt, int V) {
  if (stride < V || stride > (INT64_MAX >> 8)) return PE_EINVAL;
  return pe_host::aligned16(rows) && (stride * elt) % 16 == 0 ? PE_OK : PE_EALIGN;
}

}  // namespace

extern "C" {

int pe_draft_sample(const pe_draft_sample_args* a, void* stream) {
  if (!a) return PE_EINVAL;
  const int elt = pe_host::elt_size(a->dtype);
  if (!elt) return PE_EDTYPE;
  if (a->n < 0 || a->n > PE_MAX_SAMPLE_ROWS || a->V < 1 || a->V > PE_MAX_SAMPLE_V || a->rows < 0) return PE_EINVAL;
  if (a->n == 0) return PE_OK;
  if (a->rows < 1 || a->requests < 1 || a->n % a->requests || (!a->sample_idx && a->n > a->rows)) return PE_EINVAL;
  if (!a->logits || !a->u || !a->out_tokens || !a->err) return PE_EINVAL;
  int rc = rows_ok(a->logits, a->row_stride, elt, a->V);
  if (rc != PE_OK) return rc;
  pe_host::DeviceInfo dev;
  if (pe_host::device_info(&dev) != PE_OK) return PE_ECUDA;
  pe::FilterParams p = {};
  p.rows_a = static_cast<const char*>(a->logits);
  p.a_bytes = a->row_stride * elt;
  p.V = a->V;
  p.n = a->n;
  p.per = a->n / a->requests;
  p.src_rows = a->rows;
  p.sample_idx = a->sample_idx;
  p.asked = {a->filter.temperature, a->filter.top_k, a->filter.top_p, a->filter.min_p};
  p.u = a->u;
  p.out_tokens = a->out_tokens;
  p.out_prob = a->out_prob;
  p.err = a->err;
  split_rows(p, elt, dev.sm_count);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  rc = a->dtype == PE_BF16 ? launch_filter<PE_BF16, false>(p, st) : launch_filter<PE_F32, false>(p, st);
  return rc == PE_OK ? pe_host::launch_status() : rc;
}

size_t pe_workspace_bytes_filtered(int32_t B, int32_t Kp) {
  if (B < 0 || Kp < 0 || Kp > PE_MAX_KP) return 0;
  return FilteredLayout(B, Kp).bytes;
}

int pe_verify_filtered(const pe_verify_filtered_args* a, void* stream) {
  if (!a) return PE_EINVAL;
  const int elt = pe_host::elt_size(a->dtype);
  if (!elt) return PE_EDTYPE;
  if (a->B < 0 || a->Kp < 0 || a->Kp > PE_MAX_KP || a->V < 1 || a->V > PE_MAX_SAMPLE_V) return PE_EINVAL;
  if (a->B == 0) return PE_OK;
  const long long rows = (long long)a->B * (2 * a->Kp + 1);
  if (rows > PE_MAX_SAMPLE_ROWS) return PE_EINVAL;
  if (!a->target_logits || !a->u_draw || !a->accepted_len || !a->bonus_token || !a->workspace || !a->err) return PE_EINVAL;
  if (a->Kp > 0 && (!a->draft_logits || !a->in_tokens || !a->u_accept)) return PE_EINVAL;
  int rc = rows_ok(a->target_logits, a->target_stride, elt, a->V);
  if (rc == PE_OK && a->Kp > 0) rc = rows_ok(a->draft_logits, a->draft_stride, elt, a->V);
  if (rc != PE_OK) return rc;
  if (!pe_host::aligned16(a->workspace)) return PE_EALIGN;
  // All CTAs of a request read its coins and its number while the first one writes: over them, they would
  // not agree on the first rejection, nor on their barriers.
  const int64_t B = a->B, n = B * a->Kp;
  const void* out[3] = {a->accepted_len, a->bonus_token, a->accept_prob};
  const int64_t out_bytes[3] = {4 * B, 4 * B, 4 * n};
  for (int o = 0; o < 3; ++o)
    if (pe_host::overlap(out[o], out_bytes[o], a->u_accept, 4 * n) || pe_host::overlap(out[o], out_bytes[o], a->u_draw, 4 * B))
      return PE_EINVAL;
  pe_host::DeviceInfo dev;
  if (pe_host::device_info(&dev) != PE_OK) return PE_ECUDA;
  pe::FilterParams p = {};
  p.rows_a = static_cast<const char*>(a->target_logits);
  p.rows_b = static_cast<const char*>(a->draft_logits);
  p.a_bytes = a->target_stride * elt;
  p.b_bytes = a->draft_stride * elt;
  p.V = a->V;
  p.n = (int)rows;
  p.na = a->B * (a->Kp + 1);
  p.Kp = a->Kp;
  p.asked = {a->filter.temperature, a->filter.top_k, a->filter.top_p, a->filter.min_p};
  p.u = a->u_draw;
  p.tokens = a->in_tokens;
  p.coins = a->u_accept;
  p.accepted = a->accepted_len;
  p.bonus = a->bonus_token;
  p.chance = a->accept_prob;
  p.cuts = static_cast<pe::RowCut*>(a->workspace);
  p.kept = reinterpret_cast<pe::Kept*>(static_cast<char*>(a->workspace) + FilteredLayout(a->B, a->Kp).kept_off);
  p.err = a->err;
  split_rows(p, elt, dev.sm_count);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  rc = a->dtype == PE_BF16 ? launch_verify<PE_BF16>(p, a->B, elt, dev.sm_count, st)
                           : launch_verify<PE_F32>(p, a->B, elt, dev.sm_count, st);
  return rc == PE_OK ? pe_host::launch_status() : rc;
}

}  // extern "C"
