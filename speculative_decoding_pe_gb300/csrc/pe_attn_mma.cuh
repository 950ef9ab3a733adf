// Attention on the tensor cores (tcgen05), shared by the prompt kernel and the
// many-row kernel over the 4-bit cache.
//
// Mathematics.  For 128 rows at a time (a row is one query head of one token;
// the G heads that share a key head are stacked, so keys and values are read
// once for all of them) and 128 keys at a time:
//   S = Q K^T (fp32);  m' = max(m, max S);  P = 2^(S scale log2 e - m');
//   l = l 2^(m - m') + sum P;  O = O 2^(m - m') + P V;  out = O / l.
// O is rescaled only when the maximum grew by more than 2^8 (any m' within that
// of the true maximum gives the same quotient; P stays in range).  S, O, m and
// l are fp32.  P is rounded to the type of V for the product: 2^-9 of each
// weight on average nothing, at most as much as the rounding of the output.
//
// Work.  An item is (request, key head, up to 256 rows); its unit is a tile of
// 128 keys.  All units of the call are one line that the CTAs cut into equal
// parts, whatever the lengths are: a CTA finds its part by itself from the
// segment lengths.  An item that is cut leaves one partial (O, m, l) per CTA in
// the workspace, and whichever CTA finishes last adds them in a fixed order, so
// results do not depend on timing.
//
// CTA.  Two streams of 128 rows, one per softmax warpgroup, alternate on the
// tensor core: while one takes its exponentials, the other's products run.
// Warps 0-3 and 4-7 hold one row per thread (S and O arrive from TMEM without
// any exchange between threads), one warp issues the products, the others
// bring keys and values.
#pragma once

#include "pe_attn_line.cuh"
#include "pe_umma.cuh"

namespace pe {

constexpr float kRescale = 8.0f;  // log2 of how far P may exceed 1

// What one stream does in a segment: its visits, in order.
struct Visits {
  int count, tile0, step;
  __device__ int tile(int i) const { return tile0 + i * step; }
};
template <bool kCached>
__device__ __forceinline__ Visits visits(const Line<kCached>& line, const Walk& w, int s) {
  if (line.halves(w.rows)) {  // every other tile
    const int n = w.t1 - w.t0 - s;
    return {n > 0 ? (n + 1) / 2 : 0, w.t0 + s, 2};
  }
  const int from = w.mt * 2 * line.span + s * line.span;  // the stream's first token
  if (from >= w.rows) return {0, w.t0, 1};
  int last = w.t1;
  if (!kCached) last = min(last, (min(w.rows, from + line.span) + kTile - 1) / kTile);
  return {max(0, last - w.t0), w.t0, 1};
}

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
  static constexpr int kQ = 0;
  static constexpr int kK = 2 * kOperand;
  static constexpr int kV = kK + kStages * kOperand;
  static constexpr int kData = kV + kStages * kOperand;  // bytes, 1024-byte aligned parts
  // tensor memory: S (P takes its first half) of both streams, then O
  static constexpr int kColumns = 512;
  __host__ __device__ static constexpr uint32_t s_col(int s) { return s * kTile; }
  __host__ __device__ static constexpr uint32_t o_col(int s) { return 2 * kTile + s * D; }
};

template <int kStages>
struct AttnControl {
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_ready[kStages], v_empty[kStages];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], pair;
  Walk start;
  long long total, parts;
  uint32_t tmem;
  int dead, last[2];
  uint32_t not_finite[8][12];  // values of a masked tile: tokens that hold an infinity or NaN
  float row_scale[2][2][kTile];  // kCached, [segment parity]: the power of two taken out of a query row

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
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 4);
      mbar_init(&o_full[s], 1);
    }
    mbar_init(&pair, 8);
    dead = 0;
    mbar_init_fence();
  }
};

// ------------------------------------------------------------------- products
// The one thread that issues the tensor-core products.
template <int D, bool kCached, class Control>
__device__ void issue_products(const Line<kCached>& line, Control& c, uint32_t smem) {
  using S = AttnShape<D, kCached>;
  constexpr uint32_t kIdescS = umma_idesc(!kCached, kTile, false);
  constexpr uint32_t kIdescO = umma_idesc(!kCached, D, true);
  volatile int* dead = &c.dead;
  const uint32_t tmem = c.tmem;
  Walk w = c.start;
  uint32_t kv0 = 0, np[2] = {0, 0}, nq[2] = {0, 0};
  while (walk_next(line, w)) {
    Visits v[2] = {visits(line, w, 0), visits(line, w, 1)};
    const bool alone = line.halves(w.rows) || !v[1].count;  // a tile has one user

    auto scores = [&](int s, int i) {
      const uint32_t k = kv0 + v[s].tile(i) - w.t0, st = k % S::kStages;
      if (!wait_or_dead(&c.k_full[st], (k / S::kStages) & 1, dead)) return false;
      tc_fence_after();
      const uint32_t qa = smem + S::kQ + s * S::kOperand, ka = smem + S::kK + st * S::kOperand;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        const uint32_t off = (x / 4) * (kTile * 128) + (x % 4) * 32;
        umma_ss(tmem + S::s_col(s), umma_desc(qa + off, 16), umma_desc(ka + off, 16), kIdescS, x > 0);
      }
      tc_commit(&c.s_full[s]);
      if (alone || s == 1) tc_commit(&c.k_empty[st]);
      if (i == v[s].count - 1) tc_commit(&c.q_empty[s]);
      return true;
    };

    for (int s = 0; s < 2; ++s)
      if (v[s].count) {
        if (!wait_or_dead(&c.q_full[s], nq[s]++ & 1, dead) || !scores(s, 0)) return;
      }
    const int n = max(v[0].count, v[1].count);
    for (int i = 0; i < n; ++i)
      for (int s = 0; s < 2; ++s) {
        if (i >= v[s].count) continue;
        const uint32_t k = kv0 + v[s].tile(i) - w.t0, st = k % S::kStages;
        if (!wait_or_dead(&c.v_ready[st], (k / S::kStages) & 1, dead)) return;
        if (!wait_or_dead(&c.p_full[s], np[s]++ & 1, dead)) return;
        tc_fence_after();
        const uint32_t va = smem + S::kV + st * S::kOperand;
#pragma unroll
        for (int x = 0; x < kTile / 16; ++x)
          umma_ts(tmem + S::o_col(s), tmem + S::s_col(s) + x * 8,
                  umma_desc(va + x * 16 * 128, kTile * 128), kIdescO, i > 0 || x > 0);
        tc_commit(&c.o_full[s]);
        if (alone || s == 1) tc_commit(&c.v_empty[st]);
        if (i + 1 < v[s].count && !scores(s, i + 1)) return;
      }
    kv0 += w.t1 - w.t0;
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
};

// A partial result in the workspace: fp32 sums as float4 [D/4][256 rows], then
// (maximum, total) [256 rows].  Slots 0 and 1 of a CTA hold the items that its
// part begins and ends in, slot 2 what the two halves of an item exchange.
template <int D>
__device__ __forceinline__ float4* partial(uint8_t* ws, int cta, int slot) {
  return reinterpret_cast<float4*>(ws + AttnWorkspace::kPartials +
                                   (3LL * cta + slot) * AttnWorkspace::partial_bytes(D));
}
template <int D>
__device__ __forceinline__ void put_partial(float4* to, int row, const float (&o)[D], float m, float l) {
#pragma unroll
  for (int d = 0; d < D / 4; ++d)
    to[d * 256 + row] = make_float4(o[4 * d], o[4 * d + 1], o[4 * d + 2], o[4 * d + 3]);
  reinterpret_cast<float2*>(to + D / 4 * 256)[row] = make_float2(m, l);
}
// (o, m, l) += the partial result.
template <int D>
__device__ __forceinline__ void add_partial(const float4* from, int row, float (&o)[D], float& m, float& l) {
  const float2 ml = __ldcg(reinterpret_cast<const float2*>(from + D / 4 * 256) + row);
  if (ml.x == -INFINITY) return;  // saw no key
  const float mn = fmaxf(m, ml.x);
  const float f = m == -INFINITY ? 0.0f : exp2_approx(m - mn), g = exp2_approx(ml.x - mn);
  const bool had = m != -INFINITY;
  l = (had ? l * f : 0.0f) + ml.y * g;
  m = mn;
#pragma unroll
  for (int d = 0; d < D / 4; ++d) {
    const float4 x = __ldcg(from + d * 256 + row);
    o[4 * d] = (had ? o[4 * d] * f : 0.0f) + x.x * g;
    o[4 * d + 1] = (had ? o[4 * d + 1] * f : 0.0f) + x.y * g;
    o[4 * d + 2] = (had ? o[4 * d + 2] * f : 0.0f) + x.z * g;
    o[4 * d + 3] = (had ? o[4 * d + 3] * f : 0.0f) + x.w * g;
  }
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
  // an f16 weight loses its low end below 2^-14: the maximum is held at 2^7 (at
  // most 2^15 before a rescale), so weights down to 2^-21 of it keep every bit
  constexpr float kLift = kCached ? 7.0f : 0.0f;
  volatile int* dead = &c.dead;
  const int row = threadIdx.x & (kTile - 1);
  const uint32_t lane_base = c.tmem + ((uint32_t)(row & ~31) << 16);
  const uint32_t s_addr = lane_base + Sh::s_col(s), o_addr = lane_base + Sh::o_col(s);
  const int tok = row / line.G, g = row - tok * line.G;
  uint32_t visit = 0, filled = 0, joins = 0;  // visits, segments with visits, joins so far
  int segment = 0;
  Walk w = c.start;
  for (; walk_next(line, w); ++segment) {
    const Visits v = visits(line, w, s);
    const bool halves = line.halves(w.rows);
    const int from = halves ? 0 : (2 * w.mt + s) * line.span;
    const bool valid = tok < line.span && from + tok < w.rows;
    const int t = w.first + from + tok;
    // a row that sees nothing computes what it likes and is thrown away
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
    float m = -INFINITY, l = 0.0f, scale = p.scale_log2;
    for (int i = 0; i < v.count; ++i, ++visit) {
      if (!wait_warp(&c.s_full[s], visit & 1, dead)) return;
      tc_fence_after();
      if (kCached && i == 0) scale = p.scale_log2 * c.row_scale[filled++ & 1][s][row];
      const int key0 = v.tile(i) * kTile;
      uint32_t x[kTile];
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_ld32(s_addr + 32 * q, x + 32 * q);
      tc_wait_ld();
      if (__any_sync(0xffffffffu, limit < key0 + kTile)) {
        const int seen = limit - key0;
#pragma unroll
        for (int q = 0; q < kTile; ++q)
          if (q >= seen) x[q] = 0xff800000u;  // whatever it was: -infinity
      }
      float mx[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) mx[q] = __uint_as_float(x[q]);
#pragma unroll
      for (int q = 4; q < kTile - 4; q += 8)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          mx[r] = max3(mx[r], __uint_as_float(x[q + r]), __uint_as_float(x[q + 4 + r]));
#pragma unroll
      for (int r = 0; r < 4; ++r) mx[r] = fmaxf(mx[r], __uint_as_float(x[kTile - 4 + r]));
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
      const bool grew = top > m + kRescale;
      if (__any_sync(0xffffffffu, grew)) {
        const float f = grew ? exp2_approx(m - top) : 1.0f;
        if (grew) m = top;
        l *= f;
        if (i > 0) {  // O of the visits before
          if (!wait_warp(&c.o_full[s], (visit - 1) & 1, dead)) return;
          tc_fence_after();
#pragma unroll
          for (int q = 0; q < D; q += 32) {
            uint32_t o[32];
            tmem_ld32(o_addr + q, o);
            tc_wait_ld();
#pragma unroll
            for (int r = 0; r < 32; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * f);
            tmem_st32(o_addr + q, o);
          }
        }
      }
      const float shift = (m == -INFINITY ? 0.0f : -m) + kLift;
      float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
      for (int q = 0; q < kTile; q += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          float2 e = fma2(make_float2(__uint_as_float(x[q + 2 * r]), __uint_as_float(x[q + 2 * r + 1])),
                          make_float2(scale, scale), make_float2(shift, shift));
          e.x = exp2_approx(e.x);
          e.y = exp2_approx(e.y);
          sum[r & 1] = add2(sum[r & 1], e);
          pk[r] = kCached ? pack_f16(e.x, e.y) : pack_bf16(e.x, e.y);
        }
        tmem_st16(s_addr + q / 2, pk);
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&c.p_full[s]);
      l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
    }
    // ---- the segment's result
    float o[D];
    if (v.count) {
      if (!wait_warp(&c.o_full[s], (visit - 1) & 1, dead)) return;
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < D; q += 32) tmem_ld32(o_addr + q, reinterpret_cast<uint32_t*>(o) + q);
      tc_wait_ld();
      tc_fence_before();
    } else {
#pragma unroll
      for (int q = 0; q < D; ++q) o[q] = 0.0f;
    }
    if (!live) m = -INFINITY, l = 0.0f;
    if (!kCached) {
      // values that are not finite were taken out of masked tiles (bring_values):
      // the rows that see them get them back
      const int first_masked = (2 * w.mt * line.span + 1) / kTile;
      for (int j = max(w.t0, first_masked); j < w.t0 + v.count; ++j)
        for (int word = 0; word < 4; ++word) {
          uint32_t bits = c.not_finite[segment & 7][(j - first_masked) * 4 + word];
          for (; bits; bits &= bits - 1) {
            const int key = j * kTile + word * 32 + __ffs(bits) - 1;
            if (!live || key >= limit) continue;
            const uint16_t* src = p.v + (w.first + key) * p.v_row + w.h * p.v_head;
#pragma unroll
            for (int d = 0; d < D; ++d) {
              const uint32_t b = src[d];
              if ((b & 0x7f80u) == 0x7f80u) o[d] += __uint_as_float(b << 16);
            }
          }
        }
    }
    const bool whole = w.t0 == 0 && w.t1 == w.tiles;
    bool finish = whole;
    const int slot_row = halves ? row : s * kTile + row;
    if (halves) {  // stream 1 hands its half to stream 0
      float4* x = partial<D>(p.ws, blockIdx.x, 2);
      const int xr = (segment & 1) * kTile + row;
      if (s == 1) {
        put_partial<D>(x, xr, o, m, l);
        if (!join_streams(c, joins)) return;
      } else {
        if (!join_streams(c, joins)) return;
        add_partial<D>(x, xr, o, m, l);
      }
    }
    if (!whole) {
      const Reach at = reach(w, c.parts, c.total);  // the first part's counter counts
      const int c0 = at.first, c1 = at.last;
      if (!halves || s == 0)
        put_partial<D>(partial<D>(p.ws, blockIdx.x, (int)blockIdx.x == c0), slot_row, o, m, l);
      if (!join_streams(c, joins)) return;
      if (threadIdx.x == 0) {
        unsigned* count = reinterpret_cast<unsigned*>(p.ws) + c0;
        const unsigned old = atom_add_acq_rel_u32(count, 1);
        if (old > (unsigned)(c1 - c0)) atomicOr(p.err, PE_ERR_WORKSPACE);
        c.last[segment & 1] = old == (unsigned)(c1 - c0);
        if (c.last[segment & 1]) *count = 0;
      }
      if (!join_streams(c, joins)) return;
      finish = c.last[segment & 1] && (!halves || s == 0);
      if (finish) {
        m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int q = 0; q < D; ++q) o[q] = 0.0f;
        for (int part = c0; part <= c1; ++part)
          add_partial<D>(partial<D>(p.ws, part, part == c0), slot_row, o, m, l);
      }
    }
    if (finish && valid && (!halves || s == 0)) {
      const float r = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);  // no key: zeros; a NaN stays
      uint4* out = reinterpret_cast<uint4*>(p.out + ((long long)t * p.Hq + w.h * line.G + g) * D);
#pragma unroll
      for (int d = 0; d < D / 8; ++d) {
        uint4 y;
        uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          yw[e] = live ? pack_bf16(o[8 * d + 2 * e] * r, o[8 * d + 2 * e + 1] * r) : 0u;
        out[d] = y;
      }
    }
  }
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
