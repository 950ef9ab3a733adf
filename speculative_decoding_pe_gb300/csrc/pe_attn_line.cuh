// How an attention call is cut among the CTAs.
//
// An item is (request, key head, a block of rows); its units are blocks of
// kUnit keys.  The units of all items form one line, request after request,
// and part c of n is units [c U / n, (c + 1) U / n): equal parts whatever the
// lengths are, but that an end less than `snap` units from an item's end moves
// there, and any end in a short item, because a piece of an item costs a CTA as much
// as some units do (one token over 4000 keys, in a graph: 17.3 us against 12.7).  No
// plan is made on the host, which does not know the lengths: every CTA sums them up for
// itself (1 to 3 us of a small call, most of it the first fetch of the instructions).
#pragma once

#include "pe_attn.cuh"
#include "pe_tma.cuh"
#include "pe_umma.cuh"

namespace pe {

constexpr int kTile = 128;        // rows of a stream; keys of a tile

// a / b, in 32 bits where they do (a 64-bit division takes some 500 cycles).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// sum_{i=1..k} ceil(i w / 128)
__device__ __forceinline__ long long sum_tiles(long long k, long long w) {
  if (k < (1 << 24) && (w & (w - 1)) == 0 && w <= kTile) {  // 1, ..., 1, 2, ..., 2, ...: 128 / w of each
    const int shift = 31 - __clz(kTile / (int)w);
    const long long q = k >> shift;
    return ((q * (q + 1) / 2) << shift) + (k - (q << shift)) * (q + 1);
  }
  // sum_{i=0..k-1} floor((a i + b) / m), with ceil(x / 128) = floor((x + 127) / 128),
  // by the known reduction: whole multiples of m out of a and b, then the points under
  // the line counted by columns instead of rows, which exchanges a and m as Euclid's
  // algorithm does
  long long n = k, m = kTile, a = w, b = w + kTile - 1, sum = 0;
  for (;;) {
    if (a >= m) {
      const long long c = quotient(a, m);
      sum += (n - 1) * n / 2 * c;
      a -= c * m;
    }
    if (b >= m) {
      const long long c = quotient(b, m);
      sum += n * c;
      b -= c * m;
    }
    const long long y = a * n + b;
    if (y < m) return sum;
    n = quotient(y, m);
    b = y - n * m;
    const long long t = m;
    m = a;
    a = t;
  }
}

// How the items of a call are laid on the line of units.  `prefix` and `keys`
// lie in shared memory.
template <bool kCached, int kUnit = kTile>
struct Line {
  Segments seg;
  int Hkv, G, span;         // span: tokens of a stream (128 / G)
  const long long* prefix;  // units before request b; [B] is the total
  const int* keys;          // kCached: keys of request b

  // Over the cache an item is one stream's rows, and both streams take it, every
  // other unit each: a batch of drafts has no more rows.  A prompt's item is two.
  __device__ int tokens() const { return kCached ? span : 2 * span; }
  // units of items 0..k-1 of one (request, head)
  __device__ long long before(long long k, int rows, int nkeys) const {
    const int w = tokens();
    if (kCached) return k * max(1, (nkeys + kUnit - 1) / kUnit);
    if (k * w <= rows) return sum_tiles(k, w);
    return (k > 1 ? sum_tiles(k - 1, w) : 0) + (rows + kUnit - 1) / kUnit;
  }
  __device__ int items(int rows) const { return (rows + tokens() - 1) / tokens(); }
  __device__ int tiles(int mt, int rows, int nkeys) const {
    const long long n = kCached ? nkeys : min((long long)rows, (mt + 1LL) * tokens());
    return (int)max(1LL, (n + kUnit - 1) / kUnit);
  }
};

// One CTA's walk over its part of the line.
struct Walk {
  int b, h, mt;          // item
  int t0, t1, tiles;     // its units [t0, t1) of `tiles`
  int rows, first;       // the request's rows and its first row
  long long u, end;      // next unit, end of the part
};

template <bool kCached, int kUnit>
__device__ __forceinline__ bool walk_next(const Line<kCached, kUnit>& line, Walk& w) {
  if (w.u >= w.end) return false;
  w.t0 = w.t1;  // the tile after the last one
  if (w.t1 >= w.tiles) {
    w.t0 = 0;
    if (++w.mt >= line.items(w.rows)) {
      w.mt = 0;
      if (++w.h >= line.Hkv) {
        w.h = 0;
        do ++w.b;
        while (line.prefix[w.b + 1] == line.prefix[w.b]);  // u < end: there is one
        w.first = line.seg.begin(w.b);
        w.rows = line.seg.end(w.b) - w.first;
      }
    }
    w.tiles = line.tiles(w.mt, w.rows, kCached ? line.keys[w.b] : 0);
  }
  w.t1 = (int)min((long long)w.tiles, w.t0 + (w.end - w.u));
  w.u += w.t1 - w.t0;
  return true;
}

// The walk's state before its first segment.
template <bool kCached, int kUnit>
__device__ Walk walk_begin(const Line<kCached, kUnit>& line, long long u, long long end) {
  Walk w;
  w.u = u, w.end = end;
  w.b = w.h = w.mt = w.t0 = w.t1 = w.tiles = w.rows = w.first = 0;
  if (u >= end) return w;
  int lo = 0, hi = line.seg.B - 1;  // the last b with prefix[b] <= u
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (line.prefix[mid] <= u) lo = mid; else hi = mid - 1;
  }
  w.b = lo;  // empty requests share their prefix with the next one, and that one is later
  w.first = line.seg.begin(w.b);
  w.rows = line.seg.end(w.b) - w.first;
  const int nkeys = kCached ? line.keys[w.b] : 0;
  const long long per_head = quotient(line.prefix[w.b + 1] - line.prefix[w.b], line.Hkv);
  long long r = u - line.prefix[w.b];
  w.h = (int)quotient(r, per_head);
  r -= w.h * per_head;
  lo = 0, hi = line.items(w.rows) - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (line.before(mid, w.rows, nkeys) <= r) lo = mid; else hi = mid - 1;
  }
  w.mt = lo;
  w.tiles = line.tiles(w.mt, w.rows, nkeys);
  w.t0 = w.t1 = (int)(r - line.before(w.mt, w.rows, nkeys));
  return w;
}

// ------------------------------------------------------------------- the plan
// Every CTA lays the line out for itself (a few loads per request) and finds
// its part.  False when the offsets are no partition of the rows.
template <bool kCached, int kUnit, class Control>
__device__ bool plan(Line<kCached, kUnit>& line, int min_units, int most_snap, Control& c, long long* prefix,
                     int* keys, long long* sums, const int32_t* positions, const uint8_t* is_rejected,
                     int table_keys, uint32_t* err) {
  const int tid = threadIdx.x, n = blockDim.x, B = line.seg.B;
  if (line.seg.offsets && !offsets_valid(line.seg.offsets, B, line.seg.T, 0)) {
    if (tid == 0 && blockIdx.x == 0) atomicOr(err, PE_ERR_OFFSETS);
    return false;
  }
  if (kCached) {  // keys of a request: the most that one of its rows sees
    int lanes = 1;
    while (lanes < 32 && 2 * lanes * B <= n) lanes *= 2;
    const int groups = n / lanes, lane = tid % lanes;
    for (int b0 = 0; b0 < B; b0 += groups) {
      const int b = b0 + tid / lanes;
      int most = 0;
      bool bad = false;
      if (b < B) {
        const int end = line.seg.end(b);
        for (int t = line.seg.begin(b) + lane; t < end; t += lanes)
          most = max(most, row_limit(positions, is_rejected, t, table_keys, bad));
      }
      for (int d = lanes >> 1; d; d >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
      if (b < B && lane == 0) keys[b] = most;
      if (bad && blockIdx.x == 0) atomicOr(err, PE_ERR_BLOCK_RANGE);
    }
    __syncthreads();
  }
  line.prefix = prefix;
  line.keys = keys;
  auto units = [&](int b) {
    const int rows = line.seg.end(b) - line.seg.begin(b);
    return rows ? line.Hkv * line.before(line.items(rows), rows, kCached ? keys[b] : 0) : 0LL;
  };
  auto items = [&](int b) {
    const int rows = line.seg.end(b) - line.seg.begin(b);
    return line.Hkv * line.items(rows);
  };
  int* counts = reinterpret_cast<int*>(sums + n);
  // sums over the requests: a run of them per thread (per lane of one warp while
  // there are few), then over the threads
  const int per = (B + n - 1) / n, used = (B + per - 1) / per;
  const int b0 = tid * per, b1 = min(B, b0 + per);
  long long mine = 0;
  if (used > 32) {
    int count = 0;
    for (int b = b0; b < b1; ++b) prefix[b + 1] = mine += units(b), count += items(b);
    sums[tid] = mine;
    counts[tid] = count;
    __syncthreads();
  }
  if (tid < 32) {
    long long run = 0;
    int count = 0;
    for (int i0 = 0; i0 < used; i0 += 32) {
      const long long x = used > 32 ? sums[i0 + tid] : b0 < B ? units(b0) : 0;
      count += used > 32 ? counts[i0 + tid] : b0 < B ? items(b0) : 0;
      long long y = x;
      for (int d = 1; d < 32; d <<= 1) {
        const long long z = __shfl_up_sync(0xffffffffu, y, d);
        if (tid >= d) y += z;
      }
      if (used > 32)
        sums[i0 + tid] = run + y - x;
      else if (b0 < B)
        prefix[b0 + 1] = y;
      run += __shfl_sync(0xffffffffu, y, 31);
    }
    count = __reduce_add_sync(0xffffffffu, count);
    if (tid == 0) {
      prefix[0] = 0;
      c.total = run;
      c.items = count;
    }
  }
  if (used > 32) {
    __syncthreads();
    for (int b = b0; b < b1; ++b) prefix[b + 1] += sums[tid];
    fence_async_shared();  // the bytes of `sums` are next written by bulk and TMA copies
    __syncthreads();
  }
  __syncwarp();
  if (tid < 2) {  // the part's begin and end
    const long long total = c.total;
    // a part below min_units would spend its time on partial results, unless it is
    // a whole item (22 tokens over 8 to 16 keys, 4 heads of 128, in a graph: 77 us in
    // parts of 16 records, 13 in parts of an item)
    const long long whole = quotient(total, min_units);
    const long long parts = max(1LL, min((long long)gridDim.x, max(whole, (long long)c.items)));
    // half a part, up where the parts are items
    const long long half = quotient(total + (c.items > whole ? 2 * parts - 1 : 0), 2 * parts);
    const long long snap = min(half, (long long)most_snap);
    long long u = min(parts, (long long)blockIdx.x + tid);
    u = quotient(u * total, parts);
    Walk w = walk_begin(line, u, total);
    if (u < total) {
      const int r = w.t0, rest = w.tiles - w.t0;
      const bool keep = w.tiles <= min_units;  // an item that is not worth a cut
      if ((r <= snap || keep) && r < rest) {
        u -= r;
        w.t0 = w.t1 = 0;
      } else if (rest <= snap || keep) {
        u += rest;
        w.t0 = w.t1 = w.tiles;
      }
    }
    const long long end = __shfl_sync(3u, u, 1);
    if (tid == 0) {
      w.u = u, w.end = end;
      c.start = w;
      c.parts = parts;
      c.snap = snap;
    }
  }
  __syncthreads();
  return true;
}

// The parts that a cut item reaches over, from the walk after its segment: those
// around the ends c U / parts that lie more than `snap` units inside it.
struct Reach {
  int first, last;
};
template <class Control>
__device__ __forceinline__ Reach reach(const Walk& w, const Control& c) {
  const long long u0 = w.u - w.t1, u1 = u0 + w.tiles;  // w.u: the unit after t1
  return {(int)quotient((u0 + c.snap + 1) * c.parts + c.total - 1, c.total) - 1,
          (int)quotient((u1 - c.snap) * c.parts - 1, c.total)};
}

// An item that was cut, and the parts that hold its partial results.
struct Cut {
  Walk w;
  Reach at;
};

// How the parts of an item become one.  Whichever CTA comes last adds them all;
// or, when every CTA of the call runs at once (`together`) and the parts are many,
// each CTA adds its share of the rows after its own part.  In a graph, one request
// over 30000 keys, one key head of 128: a token 34 us alone, 16 together; a draft 107 and
// 27.  With few parts nothing is gained (4 parts 12.4 us both ways, 9 parts 54 us alone
// and 56 together).
constexpr int kTogether = 8;
// The counter: arrivals in the low half, then CTAs that have taken their share.
//
// A partial result is there.  Does this CTA add them up now?  One thread.
template <class Control>
__device__ __forceinline__ bool arrive_part(uint8_t* ws, const Walk& w, const Reach& at, bool together, Control& c,
                                            uint32_t* err) {
  unsigned* count = reinterpret_cast<unsigned*>(ws) + at.first;
  const unsigned old = atom_add_acq_rel_u32(count, 1), want = at.last - at.first;
  if ((old & 0xffffu) > want) atomicOr(err, PE_ERR_WORKSPACE);
  if (together && want + 1 >= kTogether) {
    c.cut[c.cuts].w = w;
    c.cut[c.cuts++].at = at;
    return false;
  }
  if (old == want) *count = 0;
  return old == want;
}
// Together: are all parts there (within the limit of a wait)?  One thread.
__device__ __forceinline__ bool await_parts(uint8_t* ws, const Reach& at, uint32_t* err) {
  const unsigned* count = reinterpret_cast<const unsigned*>(ws) + at.first;
  const unsigned n = at.last - at.first + 1;
  const unsigned long long t0 = global_ns();
  for (;;) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
    if ((v & 0xffffu) >= n) return true;
    if (global_ns() - t0 > kWaitLimitNs) {
      atomicOr(err, PE_ERR_TIMEOUT);
      return false;
    }
  }
}
// Together: this CTA has seen the counter; the last one that has clears it (in
// clear_parts, so that nobody waits for the answer meanwhile).  One thread.
__device__ __forceinline__ unsigned seen_parts(uint8_t* ws, const Reach& at) {
  unsigned old;
  asm volatile("atom.relaxed.gpu.global.add.u32 %0, [%1], %2;"
               : "=r"(old)
               : "l"(reinterpret_cast<unsigned*>(ws) + at.first), "r"(0x10000u)
               : "memory");
  return old >> 16;
}
__device__ __forceinline__ void clear_parts(uint8_t* ws, const Reach& at, unsigned before) {
  if (before == (unsigned)(at.last - at.first)) reinterpret_cast<unsigned*>(ws)[at.first] = 0;
}

// A running quotient: sums, their maximum and total; and the same of more parts.
// A factor of zero takes its term out whatever that is.
template <int N>
struct Running {
  float m = -INFINITY, l = 0.0f, o[N] = {};
  __device__ __forceinline__ void add(float m2, float l2, const float (&o2)[N]) {
    const float top = fmaxf(m, m2);
    const float f = m == -INFINITY ? 0.0f : exp2_approx(m - top);
    const float g = m2 == -INFINITY ? 0.0f : exp2_approx(m2 - top);
    l = (f != 0.0f ? l * f : 0.0f) + (g != 0.0f ? l2 * g : 0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = (f != 0.0f ? o[i] * f : 0.0f) + (g != 0.0f ? o2[i] * g : 0.0f);
    m = top;
  }
  // with the lane `d` away
  __device__ __forceinline__ void add_lane(int d) {
    float o2[N];
#pragma unroll
    for (int i = 0; i < N; ++i) o2[i] = __shfl_xor_sync(0xffffffffu, o[i], d);
    const float m2 = __shfl_xor_sync(0xffffffffu, m, d), l2 = __shfl_xor_sync(0xffffffffu, l, d);
    add(m2, l2, o2);
  }
};

}  // namespace pe
