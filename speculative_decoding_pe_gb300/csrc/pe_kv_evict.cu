// Eviction from the 4-bit cache by accumulated attention weight (pe_kv_evict).
//
// A cluster of C CTAs per request and key head:
//  0. the weights' ordered forms, each CTA its share of the keys, into shared memory: one
//     read, with many loads in flight;
//  1. the weight of the lightest kept key, by three passes over them with a histogram of
//     11, 11 and 10 bits, and how many keys of exactly that weight are kept (the first ones);
//  2. the kept keys in ascending order: each warp counts its share of the keys, and lists
//     it after the others' counts;
//  3. the move, in rounds: every lane holds its piece of some keys in registers, a
//     cluster barrier (where a page stays where it is), then the stores.  A kept key never moves up, so in place
//     a round's stores overwrite only keys that this round or an earlier one has read.
// Everything is exact: integers decide, bytes are moved.
//
// 256 requests of up to 32,767 keys to 2,048, 4 heads of 128: 237 us, 42 % of the bytes' floor at the copy
// rate; the latency of scattered loads bounds it (DRAM 40 % busy).  One request of 1,040 keys: 16 us, a chain
// of steps between cluster barriers.  Half or twice the keys a CTA were slower (530 and 612 us against 428).
#include "pe_cluster.cuh"
#include "pe_kv.cuh"

namespace pe {

struct EvictParams {
  int B, Hkv, block_size, bt_width, dst_width, max_keep, sinks, recent, C;
  int room;  // keys of a CTA that its shared memory holds
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

struct alignas(16) EvictShared {  // (the keys follow, in vectors)
  uint32_t hist[2][kBins];
  uint32_t counts[2][kMaxCluster];
  uint32_t heavy[kEW], equal[kEW];
  uint32_t digit, above;
};

// Order of weights; a NaN is the lightest.
__device__ __forceinline__ uint32_t mass_key(float x) { return x == x ? ordered_bits(x) : 0u; }

template <int D>
__global__ void __launch_bounds__(kET, 2) evict_kernel(const EvictParams p) {
  using R = Record<D>;
  extern __shared__ __align__(16) unsigned char smem[];
  EvictShared& sh = *reinterpret_cast<EvictShared*>(smem);
  uint32_t* held = reinterpret_cast<uint32_t*>(smem + sizeof(EvictShared));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster_rank();
  const int pair = blockIdx.x / p.C, b = pair / p.Hkv, h = pair - b * p.Hkv;
  const int bs = p.block_size;
  const int32_t* table = p.table + (long long)b * p.bt_width;
  const int32_t* dst = p.dst + (long long)b * p.dst_width;
  // the tables' first pages along with the sizes that say how many count
  constexpr int kAhead = 4;
  int32_t page[kAhead], to_page[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    page[i] = tid + i * kET < p.bt_width ? __ldg(table + tid + i * kET) : 0;
    to_page[i] = tid + i * kET < p.dst_width ? __ldg(dst + tid + i * kET) : 0;
  }
  const int n = __ldg(p.lengths + b), keep = __ldg(p.keep + b);

  // ---- sizes and pages (every CTA of the request comes to the same answer)
  const int size = min(n, keep);
  const bool sizes_ok = n >= 0 && keep >= 0 && n <= (long long)p.bt_width * bs && size <= p.max_keep &&
                        size <= (long long)p.dst_width * bs;
  int bad = 0, same = 0;  // a page outside the cache; a page that stays where it is
  if (sizes_ok) {
    const uint32_t blocks = p.num_blocks > INT32_MAX ? 0x80000000u : (uint32_t)p.num_blocks;
    const int pages = (n + bs - 1) / bs, dst_pages = (size + bs - 1) / bs;
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int i = tid + x * kET;
      bad |= (i < pages) & ((uint32_t)page[x] >= blocks);  // (negative ids too)
      bad |= (i < dst_pages) & ((uint32_t)to_page[x] >= blocks);
      same |= (i < dst_pages) & (page[x] == to_page[x]);
    }
    for (int i = tid + kAhead * kET; i < pages; i += kET) {
      const int x = __ldg(table + i), y = i < dst_pages ? __ldg(dst + i) : 0;
      bad |= (uint32_t)x >= blocks;
      bad |= (uint32_t)y >= blocks;
      same |= (i < dst_pages) & (x == y);
    }
  }
  bad = cta_count(bad != 0);
  const bool in_place = cta_count(same != 0) != 0;
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
    const int page = bs == 16 ? j >> 4 : j / bs;
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
    // every warp a run of keys, 32 at a time
    const int run = ((per + kEW - 1) / kEW + 31) & ~31;
    const int w0 = min(j1, j0 + warp * run), w1 = min(j1, w0 + run);
    const bool fits = per <= p.room;
    if (fits) {
      // four keys a load, eight loads of a thread at once (the runs of sixteen do not cross pages)
      for (int v0 = 0; 4 * v0 < j1 - j0; v0 += 8 * kET) {
        float4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int j = j0 + 4 * (v0 + i * kET + tid);
          if (j < j1) x[i] = *reinterpret_cast<const float4*>(p.mass + slot_of(table, j));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int v = v0 + i * kET + tid;
          if (j0 + 4 * v < j1)
            reinterpret_cast<uint4*>(held)[v] =
                make_uint4(mass_key(x[i].x), mass_key(x[i].y), mass_key(x[i].z), mass_key(x[i].w));
        }
      }
    }
    auto key_of = [&](int j) { return fits ? held[j - j0] : mass_key(p.mass[slot_of(table, j)]); };
    uint32_t value = 0xffffffffu, mask = 0;
    cluster_sync();  // every CTA has started; the keys are there
    if (want > 0) {
      value = 0;
      // (two histograms in turns: that of the pass before may still be read by other CTAs)
      for (int shift = 21, bits = 11, turn = 0;; turn ^= 1) {
        uint32_t* hist = sh.hist[turn];
        for (int i = tid; i < kBins; i += kET) hist[i] = 0;
        cta_sync();
#pragma unroll 4
        for (int j = k0 + tid; j < k1; j += kET) {
          const uint32_t k = key_of(j);
          if ((k & mask) == value) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1u);
        }
        if (p.C > 1) cluster_sync();
        else cta_sync();
        // bins from the heaviest on: thread tid's four
        uint32_t c[4] = {0, 0, 0, 0};
        const int bin0 = kBins - 4 - 4 * tid;
        for (int r = 0; r < p.C; ++r) {
          const uint4 q = *reinterpret_cast<const uint4*>(p.C > 1 ? at_rank(&hist[bin0], r) : &hist[bin0]);
          c[0] += q.w, c[1] += q.z, c[2] += q.y, c[3] += q.x;
        }
        const uint32_t mine = c[0] + c[1] + c[2] + c[3];
        uint32_t pre = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t x = __shfl_up_sync(0xffffffffu, pre, o);
          if (lane >= o) pre += x;
        }
        if (lane == 31) sh.heavy[warp] = pre;
        cta_sync();
        pre -= mine;
        for (int w = 0; w < warp; ++w) pre += sh.heavy[w];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (pre < want && want <= pre + c[x]) {
            sh.digit = bin0 + 3 - x;
            sh.above = pre;
          }
          pre += c[x];
        }
        cta_sync();
        value |= sh.digit << shift;
        mask |= ((1u << bits) - 1) << shift;
        want -= sh.above;
        if (shift == 0) break;
        if (shift == 21) shift = 10, bits = 11;
        else shift = 0, bits = 10;
      }
    }
    // ---- ascending list: heavier keys, the first `want` of equal weight
    // (a warp's masks of 32 keys at a time, 32 masks in turn: one in each lane)
    auto look = [&](int t0, uint2& mine) {
      for (int i = 0; i < 32 && t0 + 32 * i < w1; ++i) {
        const int j = t0 + 32 * i + lane;
        bool heavy = j < w1, equal = false;
        if (j < w1 && j >= lo && j < hi) {
          const uint32_t k = key_of(j);
          heavy = k > value;
          equal = k == value && want > 0;
        }
        const uint32_t a = __ballot_sync(0xffffffffu, heavy), e = __ballot_sync(0xffffffffu, equal);
        if (lane == i) mine = make_uint2(a, e);
      }
    };
    uint2 first_masks = make_uint2(0u, 0u);
    uint32_t heavy = 0, equal = 0;
    for (int t0 = w0; t0 < w1; t0 += 1024) {
      uint2 m = make_uint2(0u, 0u);
      look(t0, m);
      if (t0 == w0) first_masks = m;
      heavy += __reduce_add_sync(0xffffffffu, __popc(m.x));
      equal += __reduce_add_sync(0xffffffffu, __popc(m.y));
    }
    cta_sync();
    if (lane == 0) {
      sh.heavy[warp] = heavy;
      sh.equal[warp] = equal;
    }
    cta_sync();
    uint32_t heavy_all = 0, equal_all = 0, at = 0, before = 0;  // before: equal keys
    for (int w = 0; w < kEW; ++w) {
      if (w < warp) at += sh.heavy[w], before += sh.equal[w];
      heavy_all += sh.heavy[w];
      equal_all += sh.equal[w];
    }
    if (p.C > 1) {
      if (tid < p.C) {
        *at_rank(&sh.counts[0][rank], tid) = heavy_all;
        *at_rank(&sh.counts[1][rank], tid) = equal_all;
      }
      cluster_sync();
      for (int r = 0; r < rank; ++r) {
        at += sh.counts[0][r];
        before += sh.counts[1][r];
      }
    }
    at += min(want, before);
    for (int t0 = w0; t0 < w1; t0 += 1024) {
      uint2 m = first_masks;
      if (t0 != w0) look(t0, m = make_uint2(0u, 0u));
      // equal keys of the lanes before, and how many of this lane's are kept
      uint32_t eq = __popc(m.y), pre = eq;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += x;
      }
      const uint32_t all_eq = __shfl_sync(0xffffffffu, pre, 31);
      uint32_t take = before + pre - eq >= want ? 0u : min(eq, want - (before + pre - eq));
      before += all_eq;
      for (uint32_t drop = eq - take; drop; --drop) m.y ^= 0x80000000u >> __clz(m.y);  // its last ones go
      uint32_t set = m.x | m.y, n_set = __popc(set), off = n_set;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, off, o);
        if (lane >= o) off += x;
      }
      const uint32_t all = __shfl_sync(0xffffffffu, off, 31);
      int32_t* to = kept + at + off - n_set;
      for (const int j = t0 + 32 * lane; set; set &= set - 1) *to++ = j + __ffs(set) - 1;
      at += all;
    }
  } else {
    for (int j = rank * kET + tid; j < n; j += p.C * kET) kept[j] = j;
  }
  cluster_sync();  // the list is whole (and every CTA has started)

  // ---- the move
  constexpr int kLanes = D / 16;        // of a key: 16 code bytes each
  constexpr int kU = 4;                 // keys of a lane and round
  constexpr int kKeys = 32 / kLanes;    // keys that a warp moves at once
  const int part = lane % kLanes, of = lane / kLanes;
  const bool is_v = part >= kLanes / 2, has_scales = part % (kLanes / 2) == 0;
  const int code = (is_v ? R::kV : R::kK) + (part % (kLanes / 2)) * 16;
  const int scale = is_v ? R::kVs : R::kKs;
  const int round = kKeys * kU;         // keys of a warp and round (a lane looks one up)
  const int step = round * kEW * p.C;
  long long from = -1, to = -1;
  auto look_up = [&](uint32_t i) {
    from = to = -1;
    if (lane < round && (uint32_t)i < (uint32_t)size) {
      from = slot_of(table, __ldcg(kept + i));
      to = slot_of(dst, (int)i);
      if (from == to) to = -1;
    }
  };
  const uint32_t i1 = (rank * kEW + warp) * round + lane;
  look_up(i1);
  for (uint32_t i0 = 0; i0 < (uint32_t)size; i0 += step) {
    uint4 codes[kU];
    uint2 scales[kU];
    float m[kU];
    long long at[kU];
#pragma unroll
    for (int x = 0; x < kU; ++x) {
      const long long src = __shfl_sync(0xffffffffu, from, x * kKeys + of);
      at[x] = __shfl_sync(0xffffffffu, to, x * kKeys + of);
      if (at[x] >= 0) {
        const uint8_t* rec = p.cache + (src >> 4) * (long long)R::kBytes;
        const int r = (int)(src & 15);
        codes[x] = *reinterpret_cast<const uint4*>(rec + code + r * R::kRow);
        if (has_scales) {
          const uint8_t* s = rec + scale + r * R::kScaleRow;
          if (D == 128) scales[x] = *reinterpret_cast<const uint2*>(s);
          else scales[x].x = *reinterpret_cast<const uint32_t*>(s);
        }
        if (part == 0) m[x] = p.mass[src];
      }
    }
    look_up(i1 + i0 + step);  // the next round's, while these are on their way
    if (in_place) cluster_sync();
#pragma unroll
    for (int x = 0; x < kU; ++x) {
      if (at[x] >= 0) {
        uint8_t* rec = p.cache + (at[x] >> 4) * (long long)R::kBytes;
        const int r = (int)(at[x] & 15);
        *reinterpret_cast<uint4*>(rec + code + r * R::kRow) = codes[x];
        if (has_scales) {
          uint8_t* s = rec + scale + r * R::kScaleRow;
          if (D == 128) *reinterpret_cast<uint2*>(s) = scales[x];
          else *reinterpret_cast<uint32_t*>(s) = scales[x].x;
        }
        if (part == 0) p.mass[at[x]] = m[x];
      }
    }
  }
}

}  // namespace pe

namespace {
constexpr int kMostRoom = 48 * 1024;  // keys
}

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
  // A request's sizes and pages are read by the CTAs of all its key heads, at any time up to the last one's
  // start, and the first one writes: they would not agree on what there is to keep, nor on their barriers.
  const int64_t B = a->B;
  const void* out[2] = {a->out_lengths, a->kept};
  const int64_t out_bytes[2] = {4 * B, 4 * B * a->Hkv * a->max_keep};
  const void* in[4] = {a->lengths, a->keep, a->block_table, a->dst_table};
  const int64_t in_bytes[4] = {4 * B, 4 * B, 4 * B * a->bt_width, 4 * B * a->dst_width};
  for (int o = 0; o < 2; ++o)
    for (int i = 0; i < 4; ++i)
      if (pe_host::overlap(out[o], out_bytes[o], in[i], in_bytes[i])) return PE_EINVAL;
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
  // CTAs of a cluster: so many that a share of the table's keys takes at most 64 KB (two CTAs
  // and more on an SM), and more while the pairs do not fill the GPU
  const int64_t keys = (int64_t)a->bt_width * a->block_size;
  p.C = 1;
  while (p.C < 16 && (keys > 16384 * p.C || ((int64_t)a->B * a->Hkv * p.C <= dev.sm_count && keys > 512 * p.C))) p.C *= 2;
  const int64_t share = ((keys + p.C - 1) / p.C + 15) & ~15;
  p.room = (int)(share < kMostRoom ? share : kMostRoom);  // (a larger share is read from memory each time)
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)(a->B * a->Hkv * p.C));
  auto kernel = a->D == 64 ? pe::evict_kernel<64> : pe::evict_kernel<128>;
  static std::atomic<unsigned long long> done[2];
  if (!pe_host::allow_smem(kernel, (int)sizeof(pe::EvictShared) + 4 * kMostRoom, done[a->D == 64])) return PE_ECUDA;
  static std::atomic<unsigned long long> wide[2];
  if (p.C > 8 && !pe_host::allow_wide_clusters(kernel, wide[a->D == 64])) return PE_ECUDA;
  const cudaError_t rc =
      pe_host::launch_clusters(kernel, grid, pe::kET, p.C, sizeof(pe::EvictShared) + 4 * (size_t)p.room, false, st, p);
  return rc == cudaSuccess ? pe_host::launch_status() : PE_ECUDA;
}
