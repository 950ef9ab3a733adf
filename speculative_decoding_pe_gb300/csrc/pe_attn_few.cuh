// Attention over the 4-bit cache for few rows: at most 16 rows (tokens times
// query heads per key head) of a request, as a step without drafts has them.
//
// Bound by the bytes of the cache (a row of 64 keeps 8 heads: 8 products per
// code), then by the instructions that turn codes into numbers, so the layout
// serves the conversion: S^T = K Q^T and O^T = V^T P^T on m16n8k16 products, in
// which the 16-row operand is what was just converted in registers (no trip
// through shared memory as the tcgen05 operands would take) and the 8 columns
// are the rows: 8 rows fill it, where a product with the rows as M would leave
// half of it empty.  The order of elements within a product is free as long as
// both operands agree, so a lane takes 8 or 16 consecutive bytes of a token's
// keys, and 4 or 8 of its values.
//
// Weights.  P V is a tf32 product: a weight keeps 11 bits over fp32's whole range
// (in f16 those below 2^-31 of the largest would vanish, which shows where the
// heaviest keys' values are zeros), and codes times scales (6 bits) are exact.
// K Q is an f16 product: keys are exact, and queries become f16 after a power of
// two is taken out of each row (its largest element lies in [1, 2)): elements down
// to 2^-14 of it keep their 8 bits, and what a smaller one loses is below 2^-25 of
// the largest.
//
// Work.  A part of the line is a run of records (16 keys); its CTA's 8 warps
// share a segment's records and meet at its end.  Each warp brings its records
// by bulk copies, a step ahead, through segments.  A cut part has 16 records at least
// (one token over 4000 keys, in a graph: 8 records 12.9 us, 16: 12.7, 32: 13.8, 64: 16.6).
//
// Measured (in a graph), 8 rows: 256 requests of 32 000 keys on average, 4 heads of
// 128: 1.06 ms, 4.5 TB/s of the cache, 68 % of a plain copy; issue slots 61 % busy with
// conversion, waits between dependent instructions and for the alu pipe in between
// (f16 weights, whose range is not enough, 0.92 ms; bf16 weights and values 1.10 ms;
// f16 for steps without small weights and tf32 for the others 0.99 and 1.11 ms).  One
// request of 4000 keys, 8 heads of 64: 12.7 us, of which 3 are the plan, 2 the keys, 4
// the meetings of the warps and of the parts.  With 9 to 16 rows (NB = 2) some 600
// bytes a thread (D = 64: 300) spill to local memory; it is still the faster kernel
// there (pe_attn_cached.cu).
#pragma once

#include "pe_attn_line.cuh"
#include "pe_tma.cuh"
#include "pe_umma.cuh"

namespace pe {

template <int D>
struct FewShape {
  static constexpr int kWarps = 8;
  static constexpr int kStages = 2;  // (8 bits of ok_bits each)
  static constexpr int kRecords = 256 / D;                        // of a step
  static constexpr int kStep = kRecords * Record<D>::kBytes;      // 4608 bytes
  static constexpr int kRing = kWarps * kStages * kStep;
  static constexpr int kMeet = kWarps * 8 * 64 * 4;               // 64 sums of 8 rows per warp
  static constexpr int kBytes = kRing + kMeet;                    // then prefix and keys
  static constexpr int kMinRecords = 16;                          // of a part
};

template <int kWarps, int kStages>
struct FewControl {
  uint64_t full[kWarps][kStages];
  Walk start;
  long long total, parts, snap;
  int items;
  int dead, last, cuts;
  Cut cut[2];
  float m[kWarps][16], l[kWarps][16];
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], float a0, float a1, float a2, float a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)),
        "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t to_tf32(float x) {  // to nearest
  uint32_t d;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(d) : "f"(x));
  return d;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Elements 2c, 2c + 1 of row r of an 8 x 8 matrix of words (lane 4 r + c) become
// rows 2c, 2c + 1 of column r: the halves of the words are turned apart.
__device__ __forceinline__ void transpose8x8(uint32_t (&x)[2]) {
  const uint32_t lo = transpose8x8(__byte_perm(x[0], x[1], 0x5410)), hi = transpose8x8(__byte_perm(x[0], x[1], 0x7632));
  x[0] = __byte_perm(lo, hi, 0x5410), x[1] = __byte_perm(lo, hi, 0x7632);
}
template <int D, int NB>
__global__ void __launch_bounds__(256, 2) attn_few_kernel(const CachedParams p) {
  using R = Record<D>;
  using F = FewShape<D>;
  constexpr int kGroups = D / 64;       // key groups of 16 elements per lane and token
  constexpr int kSteps = D / 16;        // products of a record's scores
  constexpr int kRec = F::kRecords;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ FewControl<F::kWarps, F::kStages> c;
  long long* prefix = reinterpret_cast<long long*>(smem + F::kBytes);
  int* keys = reinterpret_cast<int*>(prefix + p.seg.B + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, cc = lane & 3;
  if (lane < F::kStages) mbar_init(&c.full[warp][lane], 1);
  if (threadIdx.x == 0) c.dead = c.cuts = 0;
  mbar_init_fence();
  Line<true, 16> line{p.seg, p.Hkv, p.Hq / p.Hkv, kTile / (p.Hq / p.Hkv), nullptr, nullptr};
  if (!plan(line, F::kMinRecords, F::kMinRecords / 2, c, prefix, keys, reinterpret_cast<long long*>(smem),
            p.positions, p.is_rejected, p.table_keys, p.err))
    return;
  if (c.start.u >= c.start.end) return;

  uint8_t* ring = smem + warp * F::kStages * F::kStep;
  float* meet = reinterpret_cast<float*>(smem + F::kRing);
  const int per_page = p.block_size >> 4;
  // the token of a record that row r of a 16-row operand holds (and r + 8: 8
  // more), so that the lanes of one load reach different banks
  constexpr uint32_t kOrder = D == 64 ? 0x57463120u : 0x67542310u;
  auto order = [&](int i) { return (int)(kOrder >> (4 * i)) & 15; };
  const int key_tok = order(r), val_a = order(2 * cc), val_b = order(2 * cc + 1);

  // ---- the loader: this warp's records in batches of 32, a lane for each; the
  // pages of the next batch are looked up while this one's copies are issued
  Walk lw = c.start;
  int lpos = 0, lend = 0;                       // what is left of the warp's share of lw
  int next_n = 0, next_rec = 0, page = -1;      // the next batch; page: this lane's
  int cur = 0, batch = 0;                       // the batch at hand: issued, in all
  uint32_t batch_ok = 0;
  const uint8_t* src = nullptr;                 // this lane's record
  uint32_t issued = 0, taken = 0, ok_bits = 0;
  auto look_up = [&]() {
    next_n = 0;
    while (lpos >= lend) {
      if (!walk_next(line, lw)) return;
      const int n = lw.t1 - lw.t0;
      lpos = lw.t0 + n * warp / F::kWarps;
      lend = lw.t0 + n * (warp + 1) / F::kWarps;
    }
    next_n = min(32, lend - lpos);
    next_rec = lpos + lane;
    page = -1;
    if (lane < next_n && next_rec * 16 < keys[lw.b])
      page = __ldg(p.block_table + (long long)lw.b * p.bt_width + next_rec / per_page);
    lpos += next_n;
  };
  auto issue = [&]() {  // the copies of one step
    if (cur >= batch) {
      if (!next_n) return;
      const bool ok = page >= 0 && page < p.num_blocks;
      if (!ok && lane < next_n && next_rec * 16 < keys[lw.b]) atomicOr(p.err, PE_ERR_BLOCK_RANGE);
      batch_ok = __ballot_sync(0xffffffffu, ok && lane < next_n);
      src = p.cache + (((long long)page * p.Hkv + lw.h) * per_page + next_rec % per_page) * R::kBytes;
      cur = 0, batch = next_n;
      look_up();
    }
    const uint32_t st = issued % F::kStages;
    const uint32_t bits = (batch_ok >> cur) & ((1u << kRec) - 1);
    ok_bits = (ok_bits & ~(0xffu << (8 * st))) | bits << (8 * st);
    if (lane == 0) mbar_arrive_expect_tx(&c.full[warp][st], __popc(bits) * R::kBytes);
    __syncwarp();
    if (lane >= cur && lane < cur + kRec && (batch_ok >> lane & 1))
      bulk_load(ring + st * F::kStep + (lane - cur) * R::kBytes, src, R::kBytes, &c.full[warp][st]);
    cur += kRec;
    ++issued;
  };
  look_up();
#pragma unroll 1
  for (int i = 0; i < F::kStages; ++i) issue();

  // partial results: [slot][row][D] sums, then (maximum, total) [row]
  auto slot = [&](int part, int i) {
    return reinterpret_cast<float*>(p.ws + AttnWorkspace::kPartials) + (2LL * part + i) * (16 * (D + 2));
  };
  auto part_of = [&](const Reach& at, int part, int row, int d, float(&x)[2]) {
    const float* from = slot(part, part == at.first);
    const float2 y = __ldcg(reinterpret_cast<const float2*>(from + row * D + d));
    x[0] = y.x, x[1] = y.y;
    return __ldcg(reinterpret_cast<const float2*>(from + 16 * D + 2 * row));
  };
  auto finish = [&](const Walk& w, int row, int d, const Running<2>& sum) {
    const float inv = sum.l > 0.0f ? 1.0f / sum.l : (sum.l == sum.l ? 0.0f : sum.l);
    *reinterpret_cast<uint32_t*>(
        p.out + ((long long)(w.first + row / line.G) * p.Hq + w.h * line.G + row % line.G) * D + d) =
        pack_bf16(sum.o[0] * inv, sum.o[1] * inv);
  };
  Walk w = c.start;
  while (walk_next(line, w)) {
    const int G = line.G, L = keys[w.b];
    const int nrows = w.rows * G;
    // ---- queries: this lane's elements of row r (and r + 8)
    uint32_t q[NB][kSteps][2];
    float sc[NB][2];        // of rows 2 cc, 2 cc + 1
    int limit[NB][2], least = INT32_MAX;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int row = 8 * b + r;
      const bool in = row < nrows;
      uint32_t raw[2 * kSteps] = {};
      float most = 0.0f;
      if (in) {
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + ((long long)(w.first + row / G) * p.Hq + w.h * G + row % G) * D + 16 * kGroups * cc);
#pragma unroll
        for (int i = 0; i < kSteps / 2; ++i) {
          const uint4 x = __ldg(src + i);
          raw[4 * i] = x.x, raw[4 * i + 1] = x.y, raw[4 * i + 2] = x.z, raw[4 * i + 3] = x.w;
        }
      }
#pragma unroll
      for (int i = 0; i < 2 * kSteps; ++i) most = fmaxf(most, fmaxf(fabsf(bf16_lo(raw[i])), fabsf(bf16_hi(raw[i]))));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
      const float2 f = row_factor(most);
#pragma unroll
      for (int i = 0; i < 2 * kSteps; ++i) q[b][i / 2][i % 2] = pack_f16(bf16_lo(raw[i]) * f.x, bf16_hi(raw[i]) * f.x);
      bool bad = false;  // reported by the plan
      const int mine = in ? row_limit(p.positions, p.is_rejected, w.first + row / G, p.table_keys, bad) : 0;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sc[b][e] = p.scale_log2 * __shfl_sync(0xffffffffu, f.y, 4 * (2 * cc + e));
        limit[b][e] = __shfl_sync(0xffffffffu, mine, 4 * (2 * cc + e));
        // a row that sees nothing computes what it likes and is thrown away
        if (limit[b][e] > 0) least = min(least, limit[b][e]);
      }
    }
    least = min(least, __shfl_xor_sync(0xffffffffu, least, 1));
    least = min(least, __shfl_xor_sync(0xffffffffu, least, 2));
    float m[NB][2], l[NB][2], o[NB][D / 16][4];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int e = 0; e < 2; ++e) m[b][e] = -INFINITY, l[b][e] = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[b][j][e] = 0.0f;
    }

    // ---- this warp's records
    const int n = w.t1 - w.t0;
    int pos = w.t0 + n * warp / F::kWarps;
    const int end = w.t0 + n * (warp + 1) / F::kWarps;
    while (pos < end) {
      const int cnt = min(kRec, end - pos);
      const uint32_t st = taken % F::kStages;
      wait_warp(&c.full[warp][st], (taken / F::kStages) & 1, &c.dead);
      ++taken;
      const uint32_t ok = (ok_bits >> (8 * st)) & 0xffu;
      const uint8_t* step = ring + st * F::kStep;
      const bool masked = cnt < kRec || ok != (1u << kRec) - 1 || (pos + kRec) * 16 > least;
      float s[NB][kRec][4];
#pragma unroll
      for (int x = 0; x < kRec; ++x) {
        const uint8_t* rec = step + x * R::kBytes;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[b][x][e] = 0.0f;
        uint32_t kw[2][2 * kGroups], ks[2][kGroups];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int tok = key_tok + 8 * e;
          if (kGroups == 1) {
            const uint2 y = *reinterpret_cast<const uint2*>(rec + R::kK + tok * R::kRow + 8 * cc);
            kw[e][0] = y.x, kw[e][1] = y.y;
            ks[e][0] = e4m3_f16x2(rec[R::kKs + tok * R::kScaleRow + cc]);
          } else {
            const uint4 y = *reinterpret_cast<const uint4*>(rec + R::kK + tok * R::kRow + 16 * cc);
            kw[e][0] = y.x, kw[e][1] = y.y, kw[e][2 * kGroups - 2] = y.z, kw[e][2 * kGroups - 1] = y.w;
            const uint32_t both =
                e4m3x2_f16x2(*reinterpret_cast<const uint16_t*>(rec + R::kKs + tok * R::kScaleRow + 2 * cc));
            ks[e][0] = __byte_perm(both, both, 0x1010);
            ks[e][kGroups - 1] = __byte_perm(both, both, 0x3232);
          }
        }
#pragma unroll
        for (int g = 0; g < 2 * kGroups; ++g) {  // 8 codes of both tokens: two products
          uint32_t a[4], b8[4];
          e2m1x8_f16(kw[0][g], a);
          e2m1x8_f16(kw[1][g], b8);
#pragma unroll
          for (int e = 0; e < 4; ++e) a[e] = hmul2(a[e], ks[0][g / 2]), b8[e] = hmul2(b8[e], ks[1][g / 2]);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            mma_f16(s[b][x], a[0], b8[0], a[1], b8[1], q[b][2 * g][0], q[b][2 * g][1]);
            mma_f16(s[b][x], a[2], b8[2], a[3], b8[3], q[b][2 * g + 1][0], q[b][2 * g + 1][1]);
          }
        }
      }
      if (masked) {
#pragma unroll
        for (int x = 0; x < kRec; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = (pos + x) * 16 + key_tok + 8 * (e >> 1);
            const bool there = x < cnt && (ok >> x & 1);
#pragma unroll
            for (int b = 0; b < NB; ++b)
              if (!there || key >= limit[b][e & 1]) s[b][x][e] = -INFINITY;
          }
      }
      // ---- maxima: a row's are shared by the 8 lanes of its column
      bool grew = false;
      float top[NB][2];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = -INFINITY;
#pragma unroll
          for (int x = 0; x < kRec; ++x) t = max3(t, s[b][x][e], s[b][x][e + 2]);
          top[b][e] = t * sc[b][e];
          grew |= top[b][e] > m[b][e] + 8.0f;
        }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = top[b][e];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
            const bool g = t > m[b][e] + 8.0f;
            const float f = g ? exp2_approx(m[b][e] - t) : 1.0f;
            if (g) m[b][e] = t;
            l[b][e] *= f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) o[b][j][e] *= f, o[b][j][e + 2] *= f;
          }
      }
      float shift[NB][2];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) shift[b][e] = m[b][e] == -INFINITY ? 0.0f : -m[b][e];
      // ---- weights
#pragma unroll
      for (int x = 0; x < kRec; ++x) {
        if (x >= cnt) break;
        const uint8_t* rec = step + x * R::kBytes;
        uint32_t pt[NB][2][2];  // of this lane's row: [half of the record][token 2 cc, 2 cc + 1 of it]
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float e = exp2_approx(fmaf(s[b][x][2 * i + y], sc[b][y], shift[b][y]));
              l[b][y] += e;
              pt[b][i][y] = to_tf32(e);
            }
            transpose8x8(pt[b][i]);
          }
        uint32_t vw[4][kGroups], vs[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = (i & 1 ? val_b : val_a) + 8 * (i >> 1);
          const uint8_t* at = rec + R::kV + tok * R::kRow + 4 * kGroups * r;
          if (kGroups == 1) {
            vw[i][0] = *reinterpret_cast<const uint32_t*>(at);
          } else {
            const uint2 y = *reinterpret_cast<const uint2*>(at);
            vw[i][0] = y.x, vw[i][kGroups - 1] = y.y;
          }
          vs[i] = rec[R::kVs + tok * R::kScaleRow + (kGroups == 1 ? r >> 1 : r)];
          // what lies past the request's keys may be anything, a NaN too
          if (masked && ((pos + x) * 16 + tok >= L || !(ok >> x & 1))) vs[i] = 0;
        }
        // a product: 8 tokens; this lane's two of them, elements 2e and 2e + 1
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t both = e4m3x2_f16x2(vs[2 * i] | vs[2 * i + 1] << 8);
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            uint32_t va[4], vb[4];
            e2m1x8_f16(vw[2 * i][g], va);
            e2m1x8_f16(vw[2 * i + 1][g], vb);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float a[4];
              mul_f16x2_f32_by<false>(va[e], both, a[0], a[1]);
              mul_f16x2_f32_by<true>(vb[e], both, a[2], a[3]);
#pragma unroll
              for (int b = 0; b < NB; ++b)
                mma_tf32(o[b][4 * g + e], a[0], a[1], a[2], a[3], pt[b][i][0], pt[b][i][1]);
            }
          }
        }
      }
      pos += cnt;
      __syncwarp();  // the step is read: its place takes the next copies
      issue();
    }

    // ---- the 8 warps meet
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[b][e] += __shfl_xor_sync(0xffffffffu, l[b][e], d);
        if (l[b][e] != l[b][e] && m[b][e] == -INFINITY) m[b][e] = 0.0f;  // a NaN is not a row that saw no key
        if (r == 0) c.m[warp][8 * b + 2 * cc + e] = m[b][e], c.l[warp][8 * b + 2 * cc + e] = l[b][e];
      }
    __syncthreads();
    const bool whole = w.t0 == 0 && w.t1 == w.tiles;
    Reach at{0, 0};
    if (!whole) at = reach(w, c);
    float* mine = slot(blockIdx.x, (int)blockIdx.x == at.first);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = -INFINITY;
        for (int i = 0; i < F::kWarps; ++i) top = fmaxf(top, c.m[i][8 * b + 2 * cc + e]);
        const float f = m[b][e] == -INFINITY ? 0.0f : exp2_approx(m[b][e] - top);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) o[b][j][e] *= f, o[b][j][e + 2] *= f;
      }
#pragma unroll
      for (int half = 0; half < kGroups; ++half) {
        // 64 elements of 8 rows: [warp][row][64]; lane r holds elements 8 kGroups r + ...
        float* to = meet + warp * 512;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<float2*>(to + (2 * cc + e) * 64 + 8 * r + 2 * j) =
                make_float2(o[b][4 * half + j][e], o[b][4 * half + j][e + 2]);
        __syncthreads();
        {
          const int row = 8 * b + warp, pair = lane;
          // element pair of the lane that held it
          const int d = (pair / 4) * 8 * kGroups + 8 * half + 2 * (pair % 4);
          float top = -INFINITY, total = 0.0f;
          float2 sum = make_float2(0.0f, 0.0f);
          for (int k = 0; k < F::kWarps; ++k) top = fmaxf(top, c.m[k][row]);
          for (int k = 0; k < F::kWarps; ++k) {
            if (c.m[k][row] == -INFINITY) continue;
            total += c.l[k][row] * exp2_approx(c.m[k][row] - top);
            const float2 y = *reinterpret_cast<const float2*>(meet + k * 512 + (row & 7) * 64 + 2 * pair);
            sum.x += y.x, sum.y += y.y;
          }
          if (row < nrows) {
            bool bad = false;
            const bool live =
                row_limit(p.positions, p.is_rejected, w.first + row / G, p.table_keys, bad) > 0;
            if (whole) {
              const float inv = total > 0.0f ? 1.0f / total : (total == total ? 0.0f : total);
              *reinterpret_cast<uint32_t*>(
                  p.out + ((long long)(w.first + row / G) * p.Hq + w.h * G + row % G) * D + d) =
                  live ? pack_bf16(sum.x * inv, sum.y * inv) : 0u;
            } else {
              *reinterpret_cast<float2*>(mine + row * D + d) = sum;
              if (d == 0)
                *reinterpret_cast<float2*>(mine + 16 * D + 2 * row) =
                    live ? make_float2(top, total) : make_float2(-INFINITY, 0.0f);
            }
          }
        }
        __syncthreads();
      }
    }
    if (!whole) {
      if (threadIdx.x == 0) c.last = arrive_part(p.ws, w, at, p.together, c, p.err);
      __syncthreads();
      if (c.last) {
        for (int i = threadIdx.x; i < nrows * (D / 2); i += 256) {
          const int row = i / (D / 2), d = 2 * (i % (D / 2));
          Running<2> sum;
#pragma unroll 8
          for (int part = at.first; part <= at.last; ++part) {
            float x[2];
            const float2 ml = part_of(at, part, row, d, x);
            sum.add(ml.x, ml.y, x);
          }
          finish(w, row, d, sum);
        }
      }
      __syncthreads();
    }
  }
  if (p.together) {  // (as add_shares of pe_attn_mma.cuh: four parts of two elements in flight)
    const int cuts = c.cuts;
    unsigned before[2] = {};
    if (threadIdx.x == 0) {
      c.last = 1;
      for (int k = 0; k < cuts; ++k) c.last &= await_parts(p.ws, c.cut[k].at, p.err);
      for (int k = 0; k < cuts; ++k) before[k & 1] = seen_parts(p.ws, c.cut[k].at);
    }
    __syncthreads();
    constexpr int kFlight = 4;
    int from[2] = {0, 0}, n[2] = {0, 0}, most = 1;  // of each item: pairs of elements; parts
    for (int k = 0; k < 2; ++k)
      if (k < cuts && c.last) {
        const Reach& at = c.cut[k].at;
        const int parts = at.last - at.first + 1, share = blockIdx.x - at.first;
        const int all = c.cut[k].w.rows * line.G * (D / 2);
        most = max(most, parts);
        from[k] = all * share / parts;
        n[k] = all * (share + 1) / parts - from[k];
      }
    int width = 32;  // a warp's pairs at a time; 32 / width lanes each
    while (width > 1 && most * width > 32 * kFlight && (n[0] + n[1]) * (64 / width) <= (int)blockDim.x) width >>= 1;
    const int sub = lane / width, stride = 32 / width;
#pragma unroll 1
    for (int x0 = warp * width; x0 < n[0] + n[1]; x0 += F::kWarps * width) {
      const int x = x0 + (lane & (width - 1));
      const bool there = x < n[0] + n[1];
      const int k = there && x >= n[0];  // (an item that this CTA has)
      const int i = !there ? from[0] : k ? from[1] + x - n[0] : from[0] + x;
      const int row = i / (D / 2), d = 2 * (i % (D / 2));
      const Reach at = c.cut[k].at;
      Running<2> sum;
#pragma unroll 1
      for (int part0 = at.first + sub; there && part0 <= at.last; part0 += stride * kFlight) {
        float y[kFlight][2];
        float2 ml[kFlight];
#pragma unroll
        for (int e = 0; e < kFlight; ++e) ml[e] = part_of(at, min(part0 + stride * e, at.last), row, d, y[e]);
#pragma unroll
        for (int e = 0; e < kFlight; ++e) sum.add(part0 + stride * e <= at.last ? ml[e].x : -INFINITY, ml[e].y, y[e]);
      }
#pragma unroll 1
      for (int e = width; e < 32; e <<= 1) sum.add_lane(e);
      if (there && sub == 0) finish(c.cut[k].w, row, d, sum);
    }
    if (threadIdx.x == 0)
      for (int k = 0; k < cuts; ++k) clear_parts(p.ws, c.cut[k].at, before[k & 1]);
  }
  if (c.dead && threadIdx.x == 0) {  // what is still on its way arrives before the CTA leaves
    atomicOr(p.err, PE_ERR_TIMEOUT);
    const unsigned long long t0 = global_ns();
    while (global_ns() - t0 < kWaitLimitNs) {
    }
  }
}

}  // namespace pe
