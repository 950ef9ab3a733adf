// Attention on the tensor cores (tcgen05), shared by the prompt kernel and the
// many-row kernel over the 4-bit cache.
//
// Mathematics.  For 128 rows at a time (a row is one query head of one token;
// the G heads that share a key head are stacked, so keys and values are read
// once for all of them) and 128 keys at a time:
//   S = Q K^T (fp32);  m' = max(m, max S);  P = 2^(S scale log2 e - m');
//   l = l 2^(m - m') + sum P;  O = O 2^(m - m') + P V;  out = O / l.
// m need not be the maximum: any m gives the same quotient as long as P and O stay
// in range, so it is taken from an item's first tile and then only when a score
// passes it by kSlack; O is rarely rescaled.  S, O, m and l are fp32.  P is
// rounded to bf16 for the product, each weight by at most 2^-8 of itself however
// small it is (an f16 would lose the small ones), as the output is.
//
// Work.  An item is (request, key head, up to 256 rows); its unit is a tile of
// 128 keys.  All units of the call are one line that the CTAs cut into equal
// parts, whatever the lengths are: a CTA finds its part by itself from the
// segment lengths.  An item that is cut leaves one partial (O, m, l) per CTA in
// the workspace; they are added in a fixed order (pe_attn_line.cuh), so results do
// not depend on timing.
//
// CTA.  Two streams of 128 rows, one per softmax warpgroup, alternate on the
// tensor core: while one takes its exponentials, the other's products run.
// Warps 0-3 and 4-7 hold one row per thread (S and O arrive from TMEM without
// any exchange between threads), one warp issues the products, the others bring
// keys and values.
#pragma once

#include "pe_attn_line.cuh"
#include "pe_umma.cuh"

namespace pe {

// What one stream does in a segment: its visits, in order.
struct Visits {
  int count, tile0, step;
  __device__ int tile(int i) const { return tile0 + i * step; }
};
template <bool kCached>
__device__ __forceinline__ Visits visits(const Line<kCached>& line, const Walk& w, int s) {
  if (kCached) {  // every other tile
    const int n = w.t1 - w.t0 - s;
    return {n > 0 ? (n + 1) / 2 : 0, w.t0 + s, 2};
  }
  const int from = w.mt * 2 * line.span + s * line.span;  // the stream's first token
  if (from >= w.rows) return {0, w.t0, 1};
  int last = w.t1;
  if (!kCached) last = min(last, (min(w.rows, from + line.span) + kTile - 1) / kTile);
  return {max(0, last - w.t0), w.t0, 1};
}

// The visits of both streams take turns until one has no more; the x-th of all.
struct Order {
  int count[2], both, total;
  __device__ Order(const Visits& a, const Visits& b)
      : count{a.count, b.count}, both(min(a.count, b.count)), total(a.count + b.count) {}
  __device__ int stream(int x) const { return x < 2 * both ? x & 1 : count[1] > count[0]; }
  __device__ int visit(int x) const { return x < 2 * both ? x >> 1 : x - both; }
  __device__ int index(int s, int i) const { return i < both ? 2 * i + s : i + both; }
};

// ------------------------------------------------------------ packed fp32 pairs
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}

// ---------------------------------------------------------------- shared memory
template <int D, bool kCached>
struct AttnShape {
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kOperand = kTile * D * 2;  // bytes of 128 rows
  static constexpr int kQ = 0;                    // (over the cache, of both streams)
  static constexpr int kK = (kCached ? 1 : 2) * kOperand;
  static constexpr int kV = kK + kStages * kOperand;
  static constexpr int kRaw = kV + kStages * kOperand;  // records as they lie in the cache
  static constexpr int kRawStages = !kCached ? 0 : D == 64 ? 4 : 2;
  static constexpr int kData = kRaw + kRawStages * (kTile / 16) * Record<D>::kBytes;
  // Tensor memory: S in as many buffers as fit beside O of both streams.  The
  // visits take them in turn, P takes the first half of its S, and a buffer's next
  // S follows the products of its P.  With three of them (D = 64, which has as many
  // exponentials as products) the softmax finds its next S ready.
  static constexpr int kColumns = 512;
  static constexpr int kBuffers = D == 64 ? 3 : 2;
  static constexpr bool kHalves = D == 128;  // P's first half is announced
  __host__ __device__ static constexpr uint32_t s_col(int buffer) { return buffer * kTile; }
  __host__ __device__ static constexpr uint32_t o_col(int s) { return kBuffers * kTile + s * D; }
};

// Entries for what look_over_values notes of a segment, read when its result is
// stored.  Every eight segments the streams wait for each other.  Before the notes of
// segment m are written, the tile five before its first has met its weights (at most
// four stages), so one stream has come to segment m - 5, and the other has stored all
// results up to the last meeting: those up to segment m - 13.
constexpr int kNotes = 16;

template <int kStages>
struct AttnControl {
  static_assert(kStages <= 4, "see kNotes");
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_ready[kStages], v_empty[kStages];
  uint64_t q_full[2], q_empty[2], pair;
  // by visit of the stream: S runs up to three ahead of the products of P, and so
  // may one warp of the others; a phase two away would look like the awaited one
  uint64_t s_full[2][4], p_half[2][4], p_full[2][4], o_full[2][4];
  Walk start;
  long long total, parts, snap;
  int items;
  uint32_t tmem;
  int dead, last[2], there, cuts;
  Cut cut[2];
  // prompts, by segment: tokens of masked tiles whose values hold an infinity or NaN,
  // and whether there is one
  uint32_t not_finite[kNotes][12];
  int any_not_finite[kNotes];
  float row_scale[4][kTile];   // kCached, by segment: the power of two taken out of a query row
  float row_sum[4][kTile];     // kCached, by segment: the sum of a query's magnitudes
  uint32_t tile_ok[16];        // kCached: records of a tile that lie in the cache
  uint8_t tile_scale[16][4];   // kCached: the largest key scale of a tile's quarters

  // Barriers before their first use; one thread.  The counts: arrivals on
  // k_full, v_ready and q_full.
  __device__ void init(int k_count, int v_count, int q_count) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&k_full[i], k_count);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_ready[i], v_count);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&q_full[s], q_count);
      mbar_init(&q_empty[s], 1);
      for (int i = 0; i < 4; ++i) {
        mbar_init(&s_full[s][i], 1);
        mbar_init(&o_full[s][i], 1);
        mbar_init(&p_half[s][i], 4);
        mbar_init(&p_full[s][i], 4);
      }
    }
    mbar_init(&pair, 8);
    dead = cuts = 0;
    mbar_init_fence();
  }
};

// ------------------------------------------------------------------- products
// The products: one elected lane.
template <int D, bool kCached, class Control>
__device__ void issue_products(const Line<kCached>& line, Control& c, uint32_t smem) {
  using S = AttnShape<D, kCached>;
  constexpr uint32_t kIdescS = umma_idesc(!kCached, kTile, false);
  constexpr uint32_t kIdescO = umma_idesc(true, D, true);
  constexpr uint32_t kStep = S::kOperand >> 4;  // of a descriptor's address
  volatile int* dead = &c.dead;
  const uint32_t tmem = c.tmem;
  const uint64_t q_desc = umma_desc(smem + S::kQ, 16), k_desc = umma_desc(smem + S::kK, 16);
  const uint64_t v_desc = umma_desc(smem + S::kV, kTile * 128);
  Walk w = c.start;
  uint32_t kv0 = 0, u0 = 0, q_phase = 0;  // tiles and visits before the segment
  uint32_t done[2] = {0, 0};                           // visits of each stream
  while (walk_next(line, w)) {
    const Visits v[2] = {visits(line, w, 0), visits(line, w, 1)};
    const Order order(v[0], v[1]);
    const bool alone = kCached || !v[1].count;  // a tile has one user
#pragma unroll 1
    for (int s = 0; s < 2; ++s)
      if (order.count[s]) {
        if (!wait_or_dead(&c.q_full[s], (q_phase >> s) & 1, dead)) return;
        q_phase ^= 1u << s;
      }
    // P V of the x-th visit, then Q K of the one that takes its buffer next
#pragma unroll 1
    for (int x = -S::kBuffers; x < order.total; ++x) {
      if (x >= 0) {
        const int s = order.stream(x), i = order.visit(x);
        const uint32_t n = (s ? done[1] : done[0]) + i;  // of the stream's visits
        const uint32_t k = kv0 + v[0].step * i + (s ? v[1].tile0 : v[0].tile0) - w.t0, st = k % S::kStages;
        const uint32_t o = tmem + S::o_col(s), p = tmem + S::s_col((u0 + x) % S::kBuffers);
        const uint64_t va = v_desc + st * kStep;
        if (!wait_or_dead(&c.v_ready[st], (k / S::kStages) & 1, dead)) return;
        if (S::kHalves) {
          if (!wait_or_dead(&c.p_half[s][n & 3], (n >> 2) & 1, dead)) return;
          tc_fence_after();
#pragma unroll
          for (int y = 0; y < kTile / 32; ++y)
            umma_ts(o, p + y * 8, va + (y * 16 * 128 >> 4), kIdescO, i > 0 || y > 0);
        }
        if (!wait_or_dead(&c.p_full[s][n & 3], (n >> 2) & 1, dead)) return;
        tc_fence_after();
#pragma unroll
        for (int y = S::kHalves ? kTile / 32 : 0; y < kTile / 16; ++y)
          umma_ts(o, p + y * 8, va + (y * 16 * 128 >> 4), kIdescO, i > 0 || y > 0);
        tc_commit(&c.o_full[s][n & 3]);
        if (alone || s == 1) tc_commit(&c.v_empty[st]);
      }
      const int next = x + S::kBuffers;
      if (next < order.total) {
        const int s = order.stream(next), i = order.visit(next);
        const uint32_t k = kv0 + v[0].step * i + (s ? v[1].tile0 : v[0].tile0) - w.t0, st = k % S::kStages;
        const int buffer = (u0 + next) % S::kBuffers;
        const uint64_t qa = q_desc + (kCached ? 0 : s) * kStep, ka = k_desc + st * kStep;
        if (!wait_or_dead(&c.k_full[st], (k / S::kStages) & 1, dead)) return;
        tc_fence_after();
#pragma unroll
        for (int y = 0; y < D / 16; ++y) {
          const uint32_t off = ((y / 4) * (kTile * 128) + (y % 4) * 32) >> 4;
          umma_ss(tmem + S::s_col(buffer), qa + off, ka + off, kIdescS, y > 0);
        }
        tc_commit(&c.s_full[s][(s ? done[1] : done[0]) + i & 3]);
        if (alone || s == 1) tc_commit(&c.k_empty[st]);
        if (i == order.count[s] - 1) tc_commit(&c.q_empty[s]);
      }
    }
    kv0 += w.t1 - w.t0;
    u0 += order.total;
    done[0] += order.count[0], done[1] += order.count[1];
  }
}

// -------------------------------------------------------------------- softmax
struct SoftmaxArgs {
  int Hq, table_keys;
  float scale_log2;
  const int32_t* positions;    // kCached
  const uint8_t* is_rejected;  // kCached
  const uint16_t* v;           // prompts: values, for those that are not finite
  long long v_row, v_head;
  uint16_t* out;
  uint8_t* ws;
  uint32_t* err;
  int together;                // kCached
};

// A partial result in the workspace: fp32 sums as float4 [D/4][256 rows], then
// (maximum, total) [256 rows].  Slots 0 and 1 of a CTA hold the items that its
// part begins and ends in, slot 2 what the two halves of an item exchange.
template <int D>
__device__ __forceinline__ float4* partial(uint8_t* ws, int cta, int slot) {
  return reinterpret_cast<float4*>(ws + AttnWorkspace::kPartials +
                                   (3LL * cta + slot) * AttnWorkspace::partial_bytes(D));
}
// Of a partial result: a row's (maximum, total).
template <int D>
__device__ __forceinline__ float2* partial_ml(float4* of, int row) {
  return reinterpret_cast<float2*>(of + D / 4 * 256) + row;
}
// The factors by which two results join: of the first, of the second.
__device__ __forceinline__ float2 join(float& m, float& l, float2 other) {
  const float mn = fmaxf(m, other.x);  // -infinity: saw no key
  const float f = m == -INFINITY ? 0.0f : exp2_approx(m - mn);
  const float g = other.x == -INFINITY ? 0.0f : exp2_approx(other.x - mn);
  l = (f != 0.0f ? l * f : 0.0f) + (g != 0.0f ? other.y * g : 0.0f);
  m = mn;
  return make_float2(f, g);
}
// x f + y g, where a factor of zero takes its term out whatever it is.
__device__ __forceinline__ float mix(float x, float f, float y, float g) {
  return (f != 0.0f ? x * f : 0.0f) + (g != 0.0f ? y * g : 0.0f);
}

// Both streams' warps; orders their writes.  False: given up.
template <class Control>
__device__ __forceinline__ bool join_streams(Control& c, uint32_t& joins) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&c.pair);
  return wait_warp(&c.pair, joins++ & 1, &c.dead);
}

// One stream's rows: s = stream, one row per thread of its four warps.
template <int D, bool kCached, class Control>
__device__ void softmax_rows(const Line<kCached>& line, Control& c, const SoftmaxArgs& p, int s) {
  using Sh = AttnShape<D, kCached>;
  // How far (log2) a score may pass the maximum that is held before the row takes
  // the new one and O is rescaled.  O must not overflow where the quotient is finite:
  // for prompts, n keys of magnitude v give up to 2^8 n v.  Over the cache a value is
  // at most 6 * 448 and keys are below 2^31, so 2^80 still leaves room; there the room
  // spares the search for a maximum, whose bound (below) lies some 2^30 to 2^50 over the
  // scores (256 drafts: 2.16 ms; 2.21 with 2^64, 2.28 with 2^40).
  constexpr float kSlack = kCached ? 80.0f : 8.0f;
  // Columns of S in registers at a time.  Over the cache eight warps that convert
  // codes share the instruction cache with the softmax, and its shorter code is
  // worth more than fewer loads (64 drafts: 808 us in 128 columns, 392 in 64); a
  // prompt's softmax is faster unrolled (eight prompts: 2.19 ms in 64, 2.06 in 128).
  constexpr int kCols = kCached ? 64 : kTile;
  volatile int* dead = &c.dead;
  const int row = threadIdx.x & (kTile - 1);
  const uint32_t lane_base = c.tmem + ((uint32_t)(row & ~31) << 16);
  const uint32_t o_addr = lane_base + Sh::o_col(s);
  const int tok = row / line.G, g = row - tok * line.G;
  uint32_t visit = 0, joins = 0, exchanges = 0;  // so far
  int segment = 0;
  Walk w = c.start;
  uint32_t kv0 = 0, u0 = 0;  // tiles and visits before the segment
  for (; walk_next(line, w); kv0 += w.t1 - w.t0, ++segment) {
    if (!kCached && segment % (kNotes / 2) == 0 && segment > 0 && !join_streams(c, joins)) return;
    const Visits v = visits(line, w, s);
    const Order order(s ? visits(line, w, 0) : v, s ? v : visits(line, w, 1));
    const uint32_t base = u0;
    u0 += order.total;
    constexpr bool halves = kCached;  // both streams have the same rows
    const int from = (halves ? w.mt : 2 * w.mt + s) * line.span;
    const bool valid = tok < line.span && from + tok < w.rows;
    const int t = w.first + from + tok;
    // a row that sees nothing computes what it likes and is thrown away;
    // its weights may overflow, and stay in its own row
    int limit = INT32_MAX;
    bool live = valid;
    if (valid) {
      if (kCached) {
        bool bad = false;
        const int n = row_limit(p.positions, p.is_rejected, t, p.table_keys, bad);
        live = n > 0;
        if (live) limit = n;
      } else {
        limit = from + tok + 1;
      }
    }
    const int least = __reduce_min_sync(0xffffffffu, limit);
    const bool idle = kCached && !__any_sync(0xffffffffu, live);
    float m = live ? -INFINITY : 0.0f, l = 0.0f, scale = p.scale_log2, row_sum = 0.0f;
    for (int i = 0; i < v.count; ++i, ++visit) {
      const uint32_t u = base + order.index(s, i);
      const int buffer = u % Sh::kBuffers;
      const uint32_t s_addr = lane_base + Sh::s_col(buffer);  // and of P
      // (a ring of a stream's own: S is at most three visits ahead)
      if (!wait_warp(&c.s_full[s][visit & 3], (visit >> 2) & 1, dead)) return;
      tc_fence_after();
      auto announce = [&](uint64_t* bar) {  // P, as far as it is written
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
      };
      if (kCached && idle) {  // every row of the warp is thrown away: P may be anything
        if (Sh::kHalves) announce(&c.p_half[s][visit & 3]);
        announce(&c.p_full[s][visit & 3]);
        continue;
      }
      const int key0 = v.tile(i) * kTile;
      const uint32_t kv = (kv0 + v.tile(i) - w.t0) & 15;
      const uint32_t ok = kCached ? c.tile_ok[kv] : 0xffu;
      if (kCached && i == 0) {
        scale = p.scale_log2 * c.row_scale[segment & 3][row];
        row_sum = p.scale_log2 * c.row_sum[segment & 3][row];
      }
      // kCols columns of S from q on; scores that a row does not see become
      // -infinity, whatever they were.
      auto load = [&](int q, uint32_t(&y)[kCols]) {
#pragma unroll
        for (int r = 0; r < kCols; r += 32) tmem_ld32(s_addr + q + r, y + r);
        tc_wait_ld();
        if (__builtin_expect(least < key0 + q + kCols || ok != 0xffu, 0)) {
          const int seen = limit - key0 - q;
          const uint32_t there = ok >> (q / 16);
#pragma unroll
          for (int r = 0; r < kCols; ++r)
            if (r >= seen || (kCached && !(there >> (r / 16) & 1))) y[r] = 0xff800000u;
        }
      };
      uint32_t y[kCols];
      load(0, y);
      // Over the cache the largest key scale s of the tile tells in advance that no
      // score can pass the maximum by too much: |q k| <= sum |q| * 6 s.  (What a row
      // takes depends on its own scores alone.)
      bool look = true;
      if (kCached) {
        const uint32_t four = *reinterpret_cast<const uint32_t*>(c.tile_scale[kv]);
        const uint32_t two = __vmaxu4(four, four >> 16), one = __vmaxu4(two, two >> 8) & 0xffu;
        float most, unused;
        f16x2_to_f32(e4m3_f16x2(one), most, unused);
        look = __any_sync(0xffffffffu, live && !(row_sum * (6.0f * most) <= m + kSlack));
      }
      if (look) {
        float mx[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) mx[r] = -INFINITY;
#pragma unroll 1
        for (int q = 0; q < kTile; q += kCols) {
          if (q > 0) load(q, y);
#pragma unroll
          for (int r = 0; r < kCols / 2; ++r)
            mx[r & 7] = max3(mx[r & 7], __uint_as_float(y[r]), __uint_as_float(y[r + kCols / 2]));
        }
        const float top =
            fmaxf(max3(mx[0], mx[1], mx[2]), max3(max3(mx[3], mx[4], mx[5]), mx[6], mx[7])) * scale;
        const bool grew = live && top > m + kSlack;
        if (__any_sync(0xffffffffu, grew)) {
          // in two steps: one is zero below 2^-126, and O may have passed m by kSlack
          const float f = grew ? exp2_approx(0.5f * (m - top)) : 1.0f;
          if (grew) m = top;
          l = l * f * f;
          if (i > 0) {  // O of the visits before
            if (!wait_warp(&c.o_full[s][(visit - 1) & 3], ((visit - 1) >> 2) & 1, dead)) return;
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < D; q += 16) {
              uint32_t o[16];
              tmem_ld16(o_addr + q, o);
              tc_wait_ld();
#pragma unroll
              for (int r = 0; r < 16; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * f * f);
              tmem_st16(o_addr + q, o);
            }
          }
        }
        if (kCols < kTile) load(0, y);
      }
      const float shift = m == -INFINITY ? 0.0f : -m;
      float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll 1
      for (int q = 0; q < kTile; q += kCols) {
        if (q > 0) load(q, y);
#pragma unroll
        for (int half = 0; half < kCols; half += 64) {
          uint32_t pk[32];
#pragma unroll
          for (int r = 0; r < 32; ++r) {
            float2 e = fma2(make_float2(__uint_as_float(y[half + 2 * r]), __uint_as_float(y[half + 2 * r + 1])),
                            make_float2(scale, scale), make_float2(shift, shift));
            e.x = exp2_approx(e.x);
            e.y = exp2_approx(e.y);
            sum[r & 1] = add2(sum[r & 1], e);
            pk[r] = pack_bf16(e.x, e.y);
          }
          tmem_st16(s_addr + (q + half) / 2, pk);
          tmem_st16(s_addr + (q + half) / 2 + 16, pk + 16);
          if (Sh::kHalves && q + half == 0) announce(&c.p_half[s][visit & 3]);
        }
      }
      announce(&c.p_full[s][visit & 3]);
      l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
    }
    // ---- the segment's result, 32 columns at a time
    if (v.count) {
      if (!wait_warp(&c.o_full[s][(visit - 1) & 3], ((visit - 1) >> 2) & 1, dead)) return;
      tc_fence_after();
    }
    if (l != l && m == -INFINITY) m = 0.0f;  // a NaN is not a row that saw no key
    if (!live) m = -INFINITY, l = 0.0f;
    const bool whole = w.t0 == 0 && w.t1 == w.tiles;
    const int slot_row = halves ? row : s * kTile + row;
    // What meets other results is held for the power of two in its total, because m may
    // lie kSlack below its largest score: a factor of zero then takes out what is below
    // 2^-126 of the sum.
    float unit = 1.0f;
    if (kCached) {
      const int e = __float_as_uint(l) >> 23;
      if (e > 0 && e < 254) unit = __uint_as_float((254 - e) << 23), m += e - 127, l *= unit;
    }
    auto sums = [&](int q, float(&o)[32]) {
      if (v.count) {
        tmem_ld32(o_addr + q, reinterpret_cast<uint32_t*>(o));
        tc_wait_ld();
        if (kCached) {
#pragma unroll
          for (int r = 0; r < 32; ++r) o[r] *= unit;
        }
      } else {
#pragma unroll
        for (int r = 0; r < 32; ++r) o[r] = 0.0f;
      }
      if (!kCached && v.count && __builtin_expect(c.any_not_finite[segment % kNotes], 0)) {
        // values that are not finite were taken out of masked tiles
        // (look_over_values): the rows that see them get them back
        const int first_masked = (2 * w.mt * line.span + 1) / kTile;
        for (int j = max(w.t0, first_masked); j < w.t0 + v.count; ++j)
          for (int word = 0; word < 4; ++word) {
            uint32_t bits = c.not_finite[segment % kNotes][(j - first_masked) * 4 + word];
            for (; bits; bits &= bits - 1) {
              const int key = j * kTile + word * 32 + __ffs(bits) - 1;
              if (!live || key >= limit) continue;
              const uint16_t* src = p.v + (w.first + key) * p.v_row + w.h * p.v_head + q;
#pragma unroll
              for (int r = 0; r < 32; ++r) {
                const uint32_t b = src[r];
                if ((b & 0x7f80u) == 0x7f80u) o[r] += __uint_as_float(b << 16);
              }
            }
          }
      }
    };
    auto finish = [&](int q, const float(&o)[32], float inv) {
      uint4* out = reinterpret_cast<uint4*>(p.out + ((long long)t * p.Hq + w.h * line.G + g) * D + q);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        uint4 y;
        uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          yw[e] = live ? pack_bf16(o[8 * d + 2 * e] * inv, o[8 * d + 2 * e + 1] * inv) : 0u;
        out[d] = y;
      }
    };
    auto inverse = [](float l) { return l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l); };  // no key: zeros
    float4* half = partial<D>(p.ws, blockIdx.x, 2);
    // (an item of one tile is stream 0's alone: 256 drafts of up to 60 keys, 4 heads of
    // 128, in a graph 54 us against 72 with an exchange of nothing)
    const bool both = halves && w.t1 - w.t0 > 1;
    const int half_row = (exchanges & 1) * kTile + row;
    exchanges += both;
    if (halves && s == 1) {  // stream 1 hands its half to stream 0
      if (both) {
#pragma unroll 1
        for (int q = 0; q < D; q += 32) {
          float o[32];
          sums(q, o);
#pragma unroll
          for (int d = 0; d < 8; ++d)
            half[(q / 4 + d) * 256 + half_row] = make_float4(o[4 * d], o[4 * d + 1], o[4 * d + 2], o[4 * d + 3]);
        }
        *partial_ml<D>(half, half_row) = make_float2(m, l);
        if (!join_streams(c, joins)) return;
      }
    } else {
      float2 fg = make_float2(1.0f, 0.0f);
      if (both) {
        if (!join_streams(c, joins)) return;
        fg = join(m, l, __ldcg(partial_ml<D>(half, half_row)));
      }
      const float inv = inverse(l);
      float4* mine = whole ? nullptr : partial<D>(p.ws, blockIdx.x, (int)blockIdx.x == reach(w, c).first);
#pragma unroll 1
      for (int q = 0; q < D; q += 32) {
        float o[32];
        sums(q, o);
        if (both) {
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            const float4 x = __ldcg(half + (q / 4 + d) * 256 + half_row);
            o[4 * d] = mix(o[4 * d], fg.x, x.x, fg.y);
            o[4 * d + 1] = mix(o[4 * d + 1], fg.x, x.y, fg.y);
            o[4 * d + 2] = mix(o[4 * d + 2], fg.x, x.z, fg.y);
            o[4 * d + 3] = mix(o[4 * d + 3], fg.x, x.w, fg.y);
          }
        }
        if (whole) {
          if (valid) finish(q, o, inv);
        } else {
#pragma unroll
          for (int d = 0; d < 8; ++d)
            mine[(q / 4 + d) * 256 + slot_row] = make_float4(o[4 * d], o[4 * d + 1], o[4 * d + 2], o[4 * d + 3]);
        }
      }
      if (!whole) *partial_ml<D>(mine, slot_row) = make_float2(m, l);
    }
    tc_fence_before();
    if (whole) continue;
    // ---- the item is cut: the CTA that comes last adds the parts, in order
    const Reach at = reach(w, c);  // the first part's counter counts
    if (!join_streams(c, joins)) return;
    if (threadIdx.x == 0) c.last[segment & 1] = arrive_part(p.ws, w, at, kCached && p.together, c, p.err);
    if (!join_streams(c, joins)) return;
    if (!c.last[segment & 1] || !valid) continue;
    // All threads of both streams add; where these have the same rows, each takes
    // half of the columns.  The loads of a part's 32 columns go together, and those
    // of the next part with them.
    m = -INFINITY;
#pragma unroll 4
    for (int part = at.first; part <= at.last; ++part)
      m = fmaxf(m, __ldcg(partial_ml<D>(partial<D>(p.ws, part, part == at.first), slot_row)).x);
    const int q0 = halves ? s * (D / 2) : 0;
#pragma unroll 1
    for (int q = q0; q < q0 + (halves ? D / 2 : D); q += 32) {
      float o[32];
#pragma unroll
      for (int r = 0; r < 32; ++r) o[r] = 0.0f;
      l = 0.0f;
#pragma unroll 2
      for (int part = at.first; part <= at.last; ++part) {
        float4* from = partial<D>(p.ws, part, part == at.first);
        const float2 ml = __ldcg(partial_ml<D>(from, slot_row));
        float4 x[8];
#pragma unroll
        for (int d = 0; d < 8; ++d) x[d] = __ldcg(from + (q / 4 + d) * 256 + slot_row);
        const bool any = ml.x != -INFINITY;  // the others hold what they like
        const float f = any ? exp2_approx(ml.x - m) : 0.0f;
        l += any ? ml.y * f : 0.0f;
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          o[4 * d] += any ? x[d].x * f : 0.0f, o[4 * d + 1] += any ? x[d].y * f : 0.0f;
          o[4 * d + 2] += any ? x[d].z * f : 0.0f, o[4 * d + 3] += any ? x[d].w * f : 0.0f;
        }
      }
      finish(q, o, inverse(l));
    }
  }
}

// Together (pe_attn_line.cuh), all warps: this CTA's share of the items that it has
// a part of.  What other CTAs just wrote takes 0.8 us to arrive, so every warp takes
// part, and as many lanes share four columns of a row as it takes for a lane to have
// all its parts (five at most) on their way at once, or as there are.
template <int D, class Control>
__device__ void add_shares(const Line<true>& line, Control& c, const CachedParams& p) {
  constexpr int kAll = kTile * (D / 4), kFlight = 5;
  const int cuts = c.cuts;
  unsigned before[2] = {};
  if (threadIdx.x == 0) {
    c.there = 1;
    for (int k = 0; k < cuts; ++k) c.there &= await_parts(p.ws, c.cut[k].at, p.err);
    for (int k = 0; k < cuts; ++k) before[k & 1] = seen_parts(p.ws, c.cut[k].at);
  }
  __syncthreads();
  int from[2] = {0, 0}, n[2] = {0, 0}, most = 1;  // of each item: rows' columns; parts
  for (int k = 0; k < 2; ++k)
    if (k < cuts && c.there) {
      const Reach& at = c.cut[k].at;
      const int parts = at.last - at.first + 1, share = blockIdx.x - at.first;
      most = max(most, parts);
      from[k] = kAll * share / parts;
      n[k] = kAll * (share + 1) / parts - from[k];
    }
  int width = 32;  // a warp's columns at a time; 32 / width lanes each
  while (width > 1 && most * width > 32 * kFlight && (n[0] + n[1]) * (64 / width) <= (int)blockDim.x) width >>= 1;
  const int lane = threadIdx.x & 31, sub = lane / width, stride = 32 / width;
#pragma unroll 1
  for (int x0 = (threadIdx.x >> 5) * width; x0 < n[0] + n[1]; x0 += (blockDim.x >> 5) * width) {
    const int x = x0 + (lane & (width - 1));
    const bool there = x < n[0] + n[1];
    const int k = there && x >= n[0];  // (an item that this CTA has: the other entry holds nothing)
    const Cut& cut = c.cut[k];
    const int i = k ? from[1] + x - n[0] : from[0] + x, r = i & (kTile - 1), d = i / kTile;
    const int tok = r / line.G, t = cut.w.mt * line.span + tok;
    const bool mine = there && tok < line.span && t < cut.w.rows;
    Running<4> sum;
    const int last = cut.at.last;
#pragma unroll 1
    for (int part0 = cut.at.first + sub; mine && part0 <= last; part0 += stride * kFlight) {
      float2 ml[kFlight];
      float4 y[kFlight];
#pragma unroll
      for (int e = 0; e < kFlight; ++e) {
        const int part = min(part0 + stride * e, last);
        float4* of = partial<D>(p.ws, part, part == cut.at.first);
        ml[e] = __ldcg(partial_ml<D>(of, r));
        y[e] = __ldcg(of + d * 256 + r);
      }
#pragma unroll
      for (int e = 0; e < kFlight; ++e)
        sum.add(part0 + stride * e <= last ? ml[e].x : -INFINITY, ml[e].y, {y[e].x, y[e].y, y[e].z, y[e].w});
    }
#pragma unroll 1
    for (int e = width; e < 32; e <<= 1) sum.add_lane(e);
    if (mine && sub == 0) {
      const float inv = sum.l > 0.0f ? 1.0f / sum.l : (sum.l == sum.l ? 0.0f : sum.l);
      *reinterpret_cast<uint2*>(
          p.out + ((long long)(cut.w.first + t) * p.Hq + cut.w.h * line.G + (r - tok * line.G)) * D + 4 * d) =
          make_uint2(pack_bf16(sum.o[0] * inv, sum.o[1] * inv), pack_bf16(sum.o[2] * inv, sum.o[3] * inv));
    }
  }
  if (threadIdx.x == 0)
    for (int k = 0; k < cuts; ++k) clear_parts(p.ws, c.cut[k].at, before[k & 1]);
}

// Some wait gave up: every role has left its loop.  What is still on its way
// into shared memory or out of the tensor core is waited for (with a limit)
// before the CTA gives its memory back.
template <int D, bool kCached, class Control>
__device__ void leave_after_timeout(Control& c, uint32_t* err) {
  if (threadIdx.x == 0) {
    atomicOr(err, PE_ERR_TIMEOUT);
    const unsigned long long t0 = global_ns();
    while (global_ns() - t0 < kWaitLimitNs) {
    }
  }
  __syncthreads();
}

}  // namespace pe
