// Eviction from the 4-bit cache by accumulated attention weight (pe_kv_evict).
//
// A cluster of C CTAs per request and key head:
//  1. the weight of the lightest kept key, by three passes over the weights with
//     a histogram of 11, 11 and 10 bits of their ordered form, and how many keys of
//     exactly that weight are kept (the first ones);
//  2. the kept keys in ascending order, each CTA its share after the others' counts;
//  3. the move, in rounds: every lane holds its piece of some keys in registers, a
//     cluster barrier, then the stores.  A kept key never moves up, so in place
//     a round's stores overwrite only keys that this round or an earlier one has read.
// Everything is exact: integers decide, bytes are moved.
#include "pe_cluster.cuh"
#include "pe_kv.cuh"

namespace pe {

struct EvictParams {
  int B, Hkv, block_size, bt_width, dst_width, max_keep, sinks, recent, C;
  long long num_blocks;
  uint8_t* cache;
  float* mass;
  const int32_t* table;
  const int32_t* dst;
  const int32_t* lengths;
  const int32_t* keep;
  int32_t* kept;
  int32_t* out_lengths;
  uint32_t* err;
};

constexpr int kET = 512;
constexpr int kEW = kET / 32;
constexpr int kBins = 2048;

struct EvictShared {
  uint32_t hist[kBins];
  uint32_t counts[2][kMaxCluster];
  uint32_t warp[kEW + 1];
  uint32_t digit, above;
};

// Order of weights; a NaN is the lightest.
__device__ __forceinline__ uint32_t mass_key(float x) { return x == x ? ordered_bits(x) : 0u; }

// Sum over the CTA; and this thread's exclusive prefix.
__device__ __forceinline__ uint32_t block_prefix(uint32_t mine, uint32_t& total, EvictShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t pre = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, pre, o);
    if (lane >= o) pre += x;
  }
  cta_sync();
  if (lane == 31) sh.warp[warp] = pre;
  cta_sync();
  uint32_t before = 0, all = 0;
  for (int w = 0; w < kEW; ++w) {
    const uint32_t x = sh.warp[w];
    if (w < warp) before += x;
    all += x;
  }
  total = all;
  return before + pre - mine;
}

template <int D>
__global__ void __launch_bounds__(kET) evict_kernel(const EvictParams p) {
  using R = Record<D>;
  __shared__ EvictShared sh;
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = (int)cluster_rank();
  const int pair = blockIdx.x / p.C, b = pair / p.Hkv, h = pair - b * p.Hkv;
  const int bs = p.block_size;
  const int n = __ldg(p.lengths + b), keep = __ldg(p.keep + b);
  const int32_t* table = p.table + (long long)b * p.bt_width;
  const int32_t* dst = p.dst + (long long)b * p.dst_width;

  // ---- sizes and pages (every CTA of the request comes to the same answer)
  const int size = min(n, keep);
  const bool sizes_ok = n >= 0 && keep >= 0 && n <= (long long)p.bt_width * bs && size <= p.max_keep &&
                        size <= (long long)p.dst_width * bs;
  int bad = 0;
  if (sizes_ok) {
    for (int i = tid; i < (n + bs - 1) / bs; i += kET) {
      const int x = __ldg(table + i);
      bad |= x < 0 || x >= p.num_blocks;
    }
    for (int i = tid; i < (size + bs - 1) / bs; i += kET) {
      const int x = __ldg(dst + i);
      bad |= x < 0 || x >= p.num_blocks;
    }
  }
  bad = __syncthreads_or(bad);
  if (!sizes_ok || bad) {
    if (rank == 0 && h == 0 && tid == 0) {
      atomicOr(p.err, sizes_ok ? PE_ERR_BLOCK_RANGE : PE_ERR_PARAM);
      p.out_lengths[b] = -1;
    }
    return;
  }
  if (rank == 0 && h == 0 && tid == 0) p.out_lengths[b] = size;
  if (size == 0) return;
  int32_t* kept = p.kept + ((long long)b * p.Hkv + h) * p.max_keep;
  auto slot_of = [&](const int32_t* tab, int j) {  // index into mass
    const int page = j / bs;
    return ((long long)__ldg(tab + page) * p.Hkv + h) * bs + (j - page * bs);
  };

  if (n > size) {
    // ---- the lightest kept weight
    const int first = min(p.sinks, size), last = min(p.recent, size - first);
    uint32_t want = size - first - last;  // of the keys lo..hi-1
    const int lo = first, hi = n - last;
    const int per = ((n + p.C - 1) / p.C + 15) & ~15;
    const int j0 = min(n, rank * per), j1 = min(n, j0 + per);
    const int k0 = max(j0, lo), k1 = min(j1, hi);
    uint32_t value = 0, mask = 0;
    if (want > 0) {
      cluster_sync();  // every CTA has started
      for (int shift = 21, bits = 11;; ) {
        for (int i = tid; i < kBins; i += kET) sh.hist[i] = 0;
        cta_sync();
        for (int j = k0 + tid; j < k1; j += kET) {
          const uint32_t k = mass_key(p.mass[slot_of(table, j)]);
          if ((k & mask) == value) atomicAdd(&sh.hist[(k >> shift) & ((1u << bits) - 1)], 1u);
        }
        cluster_sync();
        // bins from the heaviest on: thread tid's four
        uint32_t c[4], mine = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int bin = kBins - 1 - (4 * tid + x);
          uint32_t s = 0;
          for (int r = 0; r < p.C; ++r) s += *at_rank(&sh.hist[bin], r);
          c[x] = s;
          mine += s;
        }
        uint32_t total;
        uint32_t pre = block_prefix(mine, total, sh);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (pre < want && want <= pre + c[x]) {
            sh.digit = kBins - 1 - (4 * tid + x);
            sh.above = pre;
          }
          pre += c[x];
        }
        cluster_sync();  // also: the histograms have been read
        value |= sh.digit << shift;
        mask |= ((1u << bits) - 1) << shift;
        want -= sh.above;
        if (shift == 0) break;
        if (shift == 21) shift = 10, bits = 11;
        else shift = 0, bits = 10;
      }
    } else {
      value = 0xffffffffu;  // nothing but the first and the last
    }
    // ---- ascending list: heavier keys, the first `want` of equal weight
    auto state = [&](int j) -> int {  // 2 kept, 1 equal, 0 not
      if (j < lo || j >= hi) return 2;
      const uint32_t k = mass_key(p.mass[slot_of(table, j)]);
      return k > value ? 2 : k == value && want > 0 ? 1 : 0;
    };
    uint32_t heavy = 0, equal = 0;
    for (int j = j0 + tid; j < j1; j += kET) {
      const int s = state(j);
      heavy += s == 2;
      equal += s == 1;
    }
    uint32_t heavy_all, equal_all;
    block_prefix(heavy, heavy_all, sh);
    block_prefix(equal, equal_all, sh);
    cluster_sync();
    if (tid < p.C) {
      *at_rank(&sh.counts[0][rank], tid) = heavy_all;
      *at_rank(&sh.counts[1][rank], tid) = equal_all;
    }
    cluster_sync();
    uint32_t equal_before = 0, at = 0;
    for (int r = 0; r < rank; ++r) {
      at += sh.counts[0][r] + min(sh.counts[1][r], want - min(want, equal_before));
      equal_before += sh.counts[1][r];
    }
    for (int t0 = j0; t0 < j1; t0 += kET) {
      const int j = t0 + tid;
      const int s = j < j1 ? state(j) : 0;
      uint32_t eq, all;
      const uint32_t e = block_prefix(s == 1, eq, sh);
      const bool in = s == 2 || (s == 1 && equal_before + e < want);
      const uint32_t o = block_prefix(in, all, sh);
      if (in) kept[at + o] = j;
      at += all;
      equal_before += eq;
    }
  } else {
    for (int j = rank * kET + tid; j < n; j += p.C * kET) kept[j] = j;
  }
  cluster_sync();  // the list is whole (and every CTA has started)

  // ---- the move
  constexpr int kLanes = D / 16;       // of a key: 16 code bytes each
  constexpr int kU = 4;                // keys of a lane group and round
  const int part = tid % kLanes, group = tid / kLanes;
  const int groups = kET / kLanes;
  const bool is_v = part >= kLanes / 2;
  const int code = (is_v ? R::kV : R::kK) + (part % (kLanes / 2)) * 16;
  for (int i0 = 0; i0 < size; i0 += groups * kU * p.C) {
    uint4 codes[kU];
    uint2 scales[kU];
    float m[kU];
    long long to[kU];
#pragma unroll
    for (int x = 0; x < kU; ++x) {
      const int i = i0 + (x * p.C + rank) * groups + group;
      to[x] = -1;
      if (i < size) {
        const int j = __ldcg(kept + i);
        const long long from = slot_of(table, j);
        const long long at = slot_of(dst, i);
        if (from != at) {
          to[x] = at;
          const uint8_t* rec = p.cache + (from >> 4) * (long long)R::kBytes;
          const int r = (int)(from & 15);
          codes[x] = *reinterpret_cast<const uint4*>(rec + code + r * R::kRow);
          if (part % (kLanes / 2) == 0) {
            const uint8_t* s = rec + (is_v ? R::kVs : R::kKs) + r * R::kScaleRow;
            if (D == 128) scales[x] = *reinterpret_cast<const uint2*>(s);
            else scales[x].x = *reinterpret_cast<const uint32_t*>(s);
          }
          if (part == 0) m[x] = p.mass[from];
        }
      }
    }
    cluster_sync();
#pragma unroll
    for (int x = 0; x < kU; ++x) {
      if (to[x] >= 0) {
        uint8_t* rec = p.cache + (to[x] >> 4) * (long long)R::kBytes;
        const int r = (int)(to[x] & 15);
        *reinterpret_cast<uint4*>(rec + code + r * R::kRow) = codes[x];
        if (part % (kLanes / 2) == 0) {
          uint8_t* s = rec + (is_v ? R::kVs : R::kKs) + r * R::kScaleRow;
          if (D == 128) *reinterpret_cast<uint2*>(s) = scales[x];
          else *reinterpret_cast<uint32_t*>(s) = scales[x].x;
        }
        if (part == 0) p.mass[to[x]] = m[x];
      }
    }
  }
  (void)lane;
}

}  // namespace pe

extern "C" int pe_kv_evict(const pe_kv_evict_args* a, void* stream) {
  if (!a) return PE_EINVAL;
  if (!pe_host::cache_sizes_ok(a->num_blocks, a->block_size, a->Hkv, a->D)) return PE_EINVAL;
  if (a->B < 0 || a->bt_width < 1 || a->dst_width < 1 || a->max_keep < 1 || a->sinks < 0 || a->recent < 0) return PE_EINVAL;
  if ((int64_t)a->bt_width * a->block_size > INT32_MAX || (int64_t)a->dst_width * a->block_size > INT32_MAX ||
      (int64_t)a->B * a->Hkv > (1 << 24))
    return PE_EINVAL;
  if (a->B == 0) return PE_OK;
  if (!a->cache || !a->mass || !a->block_table || !a->dst_table || !a->lengths || !a->keep || !a->kept || !a->out_lengths ||
      !a->err)
    return PE_EINVAL;
  if (!pe_host::aligned16(a->cache) || !pe_host::aligned16(a->mass)) return PE_EALIGN;
  pe_host::DeviceInfo dev;
  if (pe_host::device_info(&dev) != PE_OK) return PE_ECUDA;
  pe::EvictParams p = {};
  p.B = a->B, p.Hkv = a->Hkv, p.block_size = a->block_size, p.bt_width = a->bt_width, p.dst_width = a->dst_width;
  p.max_keep = a->max_keep, p.sinks = a->sinks, p.recent = a->recent;
  p.num_blocks = a->num_blocks;
  p.cache = static_cast<uint8_t*>(a->cache);
  p.mass = a->mass;
  p.table = a->block_table, p.dst = a->dst_table, p.lengths = a->lengths, p.keep = a->keep;
  p.kept = a->kept, p.out_lengths = a->out_lengths, p.err = a->err;
  p.C = 1;
  while (p.C < 8 && (int64_t)a->B * a->Hkv * p.C * 2 <= 4 * dev.sm_count) p.C *= 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = (unsigned)(a->B * a->Hkv * p.C);
  const cudaError_t rc =
      pe_host::launch_clusters(a->D == 64 ? pe::evict_kernel<64> : pe::evict_kernel<128>, grid, pe::kET, p.C, 0, false, st, p);
  return rc == cudaSuccess ? pe_host::launch_status() : PE_ECUDA;
}
