// Attention over the 4-bit cache for more rows than pe_attn_few.cuh takes: the
// tensor-core attention of pe_attn_mma.cuh, with its operands made from codes.
//
// One warp brings the records of a key tile as they lie in the cache (one bulk
// copy per record, ahead of their use by the ring of raw tiles), four warps turn
// key codes into operands and four value codes, one token per thread: code times
// scale has 6 bits and is exact in f16 and in bf16.  Keys and values have the same
// layout (128-byte rows of 64 elements, swizzled); the products read values with
// their contiguous axis along N.  Queries become f16 after a power of two is taken
// out of each row, which the softmax puts back into its scale (see pe_attn_few.cuh
// for what that costs).  Weights stay bf16, and so do values: an f16 weight below
// 2^-31 of the largest would vanish, which shows where the heaviest keys' values
// are zeros.
//
// Codes become operands (K 9, V 17 instructions a word of 8 codes) and scores weights
// (2.5 each) on the same issue slots.  With heads of 64 these bound it: 58 % of the slots
// are busy, the tensor cores 32 %, memory 25 %.  More converter warps, a warp of its own
// for the largest scales, or converters on two of the four schedulers each changed
// nothing: what counts is the number of instructions, and that the loops of the roles
// fit the instruction cache together.  With heads of 128 nothing is that busy (slots 50
// %, tensor cores 38 %, memory 30 %): two stages of keys, values and raw records, and
// two buffers of scores, leave the roles waiting for each other.
//
// Measured (in a graph), 14 rows (drafts) of 8 heads: 64 requests of 16 500 keys, 8 key
// heads of 64: 0.39 ms (1.6 TB/s of the cache, 0.38 PFLOP/s of rows that are not rejected
// or padding); 256 of 32 000, 4 heads of 128: 2.16 ms (2.3 TB/s, 0.54 PFLOP/s).  One
// request of 6000 keys: 18.5 us.
#pragma once

#include "pe_attn_mma.cuh"

namespace pe {

constexpr int kManyThreads = 20 * 32;
__device__ __forceinline__ void store_shared(uint32_t at, const uint32_t (&x)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3])
               : "memory");
}

constexpr int kConverters = 4;  // warps for keys, and as many for values

template <int kRawStages>
struct RawControl {
  uint64_t full[kRawStages], empty[kRawStages];
  uint32_t ok[kRawStages];  // records that came
};

// Records into the ring of raw tiles; one warp.  A lane looks up the page of one
// record of the next four tiles while the copies of these four are issued.
template <int D, class Control, class Raw>
__device__ void bring_records(const Line<true>& line, Control& c, Raw& raw, const CachedParams& p, uint8_t* smem) {
  using S = AttnShape<D, true>;
  using R = Record<D>;
  constexpr int kRecords = kTile / 16, kAhead = 32 / kRecords;
  volatile int* dead = &c.dead;
  const int lane = threadIdx.x & 31, per_page = p.block_size >> 4;
  Walk w = c.start;
  bool more = walk_next(line, w);
  int j = w.t0;  // first of the tiles ahead
  // the page of this lane's record of the tiles ahead
  auto look_up = [&]() {
    const int rec = j * kRecords + lane;
    if (!more || j + lane / kRecords >= w.t1 || rec * 16 >= line.keys[w.b]) return -1;
    return __ldg(p.block_table + (long long)w.b * p.bt_width + rec / per_page);
  };
  int ahead = look_up();
  for (uint32_t k = 0; more;) {
    const int page = ahead, rec = j * kRecords + lane, tiles = min(kAhead, w.t1 - j);
    const bool wanted = lane < tiles * kRecords && rec * 16 < line.keys[w.b];
    const uint8_t* base = p.cache + ((long long)w.h * per_page + rec % per_page) * R::kBytes;
    j += tiles;
    if (j >= w.t1) {
      more = walk_next(line, w);
      j = w.t0;
    }
    ahead = look_up();
    const bool ok = wanted && page >= 0 && page < p.num_blocks;
    if (wanted && !ok) atomicOr(p.err, PE_ERR_BLOCK_RANGE);
    const uint32_t all = __ballot_sync(0xffffffffu, ok);
    const uint8_t* src = base + (long long)page * p.Hkv * per_page * R::kBytes;
#pragma unroll 1
    for (int q = 0; q < tiles; ++q, ++k) {
      const uint32_t st = k % S::kRawStages;
      if (!wait_warp(&raw.empty[st], ((k / S::kRawStages) & 1) ^ 1, dead)) return;
      if (lane == 0) {
        raw.ok[st] = (all >> (q * kRecords)) & 0xffu;
        mbar_arrive_expect_tx(&raw.full[st], __popc(raw.ok[st]) * R::kBytes);
      }
      __syncwarp();
      if (ok && lane / kRecords == q)
        bulk_load(smem + S::kRaw + (st * kRecords + lane % kRecords) * R::kBytes, src, R::kBytes, &raw.full[st]);
    }
  }
}

// Codes of one token, D elements, into row `row` of an operand tile: as f16 (the
// keys, next to f16 queries) or as bf16 (the values, next to bf16 weights).
// Both are exact.  Values rolled, keys two steps at a time: the roles of this
// kernel share an instruction cache (64 drafts, in a graph: 392 us; values two steps
// at a time too, 395; keys rolled too, 399).
template <int D, bool kBf16, int kUnroll = kBf16 ? 1 : 2>
__device__ __forceinline__ void put_codes(uint8_t* tile, int row, const uint8_t* codes, const uint8_t* scales,
                                          bool valid) {
  // chunk c (8 elements) of a row lies at c ^ (row & 7)
  uint32_t at = smem_addr(tile) + row * 128 + (row & 7) * 16;
  uint32_t chunk = 0;
#pragma unroll kUnroll
  for (int i = 0; i < D / 32; ++i) {
    const uint4 y = reinterpret_cast<const uint4*>(codes)[i];
    // past the request's keys lies anything, a NaN too (codes are finite)
    const uint32_t two = valid ? reinterpret_cast<const uint16_t*>(scales)[i] : 0u;
    const uint32_t s[2] = {e4m3_f16x2(two & 0xffu), e4m3_f16x2(two >> 8)};
    const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // 8 elements: 16 bytes
      uint32_t x[4];
      e2m1x8_f16(w[q], x);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (kBf16) {
          float lo, hi;
          mul_f16x2_f32(x[e], s[q / 2], lo, hi);
          x[e] = pack_bf16(lo, hi);
        } else {
          x[e] = hmul2(x[e], s[q / 2]);
        }
      }
      store_shared(at ^ (chunk + q * 16), x);
    }
    chunk ^= 64;
    if (i & 1) at += kTile * 128;
  }
}

// The values of every tile, or its keys and (kKeys) the queries; `row`: this
// thread's row of a tile.
template <int D, bool kKeys, class Control, class Raw>
__device__ void convert_tiles(const Line<true>& line, Control& c, Raw& raw, const CachedParams& p, uint8_t* smem,
                              int row) {
  using S = AttnShape<D, true>;
  using R = Record<D>;
  volatile int* dead = &c.dead;
  const int tok = row / line.G, g = row - tok * line.G;
  const bool first_lane = (threadIdx.x & 31) == 0;
  Walk w = c.start;
  uint32_t k = 0, used[2] = {0, 0};  // tiles; segments that each stream visited
  bool busy[2] = {false, false};     // it may still read the queries there
  for (int segment = 0; walk_next(line, w); ++segment) {
    if (kKeys) {
      // this row's query, its largest element brought to [1, 2)
      const int t = w.mt * line.span + tok;
      const bool valid = tok < line.span && t < w.rows;
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + ((long long)(w.first + t) * p.Hq + w.h * line.G + g) * D);
      float most = 0.0f, all = 0.0f;
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        const uint4 q = valid ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
        const uint32_t y[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          most = fmaxf(most, fmaxf(fabsf(bf16_lo(y[e])), fabsf(bf16_hi(y[e]))));
          all += fabsf(bf16_lo(y[e])) + fabsf(bf16_hi(y[e]));
        }
      }
      const float2 f = row_factor(most);
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (busy[s] && !wait_warp(&c.q_empty[s], (used[s] - 1) & 1, dead)) return;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        busy[s] = visits(line, w, s).count > 0;
        used[s] += busy[s];
      }
      c.row_scale[segment & 3][row] = f.y;
      c.row_sum[segment & 3][row] = all * 1.001f;  // (a bound: its own roundings)
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        const uint4 q = valid ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
        uint32_t y[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = pack_f16(bf16_lo(y[e]) * f.x, bf16_hi(y[e]) * f.x);
        *reinterpret_cast<uint4*>(smem + S::kQ + (i / 8) * kTile * 128 + row * 128 + ((i % 8) ^ (row & 7)) * 16) =
            make_uint4(y[0], y[1], y[2], y[3]);
      }
      fence_async_shared();
      __syncwarp();
      if (first_lane)
        for (int s = 0; s < 2; ++s)
          if (busy[s]) mbar_arrive(&c.q_full[s]);
    }
    const int keys = line.keys[w.b];
    for (int j = w.t0; j < w.t1; ++j, ++k) {
      const uint32_t st = k % S::kStages, phase = (k / S::kStages) & 1, rst = k % S::kRawStages;
      if (!wait_warp(&raw.full[rst], (k / S::kRawStages) & 1, dead)) return;
      const uint8_t* rec = smem + S::kRaw + (rst * (kTile / 16) + row / 16) * R::kBytes;
      const int r = row & 15;
      const uint32_t ok = raw.ok[rst];
      const bool valid = j * kTile + row < keys && (ok >> (row / 16) & 1);
      const uint8_t* scales = rec + (kKeys ? R::kKs : R::kVs) + r * R::kScaleRow;
      uint32_t most = 0;  // the largest scale of the warp's keys (the bytes of magnitudes are in order)
      if (kKeys) {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) most = __vmaxu4(most, reinterpret_cast<const uint32_t*>(scales)[i] & 0x7f7f7f7fu);
        most = __vmaxu4(most, most >> 16);
        most = __reduce_max_sync(0xffffffffu, valid ? __vmaxu4(most, most >> 8) & 0xffu : 0u);
      }
      if (!wait_warp(kKeys ? &c.k_empty[st] : &c.v_empty[st], phase ^ 1, dead)) return;
      if (kKeys && first_lane) c.tile_scale[k & 15][row / 32] = (uint8_t)most;
      if (kKeys && row == 0)
        c.tile_ok[k & 15] = ok | ~((1u << min(kTile / 16, (keys - j * kTile + 15) / 16)) - 1) & 0xffu;
      put_codes<D, !kKeys>(smem + (kKeys ? S::kK : S::kV) + st * S::kOperand, row,
                           rec + (kKeys ? R::kK : R::kV) + r * R::kRow, scales, valid);
      fence_async_shared();
      __syncwarp();
      if (first_lane) {
        mbar_arrive(kKeys ? &c.k_full[st] : &c.v_ready[st]);
        mbar_arrive(&raw.empty[rst]);
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kManyThreads, 1) attn_many_kernel(const CachedParams p) {
  using S = AttnShape<D, true>;
  extern __shared__ uint8_t raw_smem[];
  __shared__ AttnControl<S::kStages> c;
  __shared__ RawControl<S::kRawStages> raw;
  uint8_t* smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  long long* prefix = reinterpret_cast<long long*>(smem + S::kData);
  int* keys = reinterpret_cast<int*>(prefix + p.seg.B + 1);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kRawStages; ++i) {
      mbar_init(&raw.full[i], 1);
      mbar_init(&raw.empty[i], 2 * kConverters);
    }
    c.init(kConverters, kConverters, kConverters);
  }
  const int G = p.Hq / p.Hkv;
  Line<true> line{p.seg, p.Hkv, G, kTile / G, nullptr, nullptr};
  if (!plan(line, 2, 2, c, prefix, keys, reinterpret_cast<long long*>(smem), p.positions, p.is_rejected, p.table_keys,
            p.err))
    return;
  if (c.start.u >= c.start.end) return;  // fewer parts than CTAs
  if (warp == 8) tmem_alloc(&c.tmem, S::kColumns);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // 20 warps of 96 registers: 128 for the softmax's rows, 72 for the products,
  // the loads and the converters
  if (warp < 8)
    take_registers<128>();
  else
    give_registers<72>();
  if (warp < 8) {
    SoftmaxArgs a;
    a.Hq = p.Hq, a.table_keys = p.table_keys, a.scale_log2 = p.scale_log2;
    a.positions = p.positions, a.is_rejected = p.is_rejected;
    a.v = nullptr, a.v_row = a.v_head = 0;
    a.out = p.out, a.ws = p.ws, a.err = p.err, a.together = p.together;
    softmax_rows<D, true>(line, c, a, warp >> 2);
  } else if (warp == 8) {
    if (elect_one()) issue_products<D, true>(line, c, smem_addr(smem));
  } else if (warp == 9) {
    bring_records<D>(line, c, raw, p, smem);
  } else if (warp >= 12 + kConverters) {
    convert_tiles<D, false>(line, c, raw, p, smem, threadIdx.x - (12 + kConverters) * 32);
  } else if (warp >= 12) {
    convert_tiles<D, true>(line, c, raw, p, smem, threadIdx.x - 12 * 32);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (p.together) {
    // as many registers as the compiler counts on: the softmax gives back first
    if (warp < 8)
      give_registers<96>();
    else
      take_registers<96>();
    if (!c.dead) add_shares<D>(line, c, p);
  }
  if (c.dead) leave_after_timeout<D, true>(c, p.err);
  if (warp == 8) tmem_dealloc(c.tmem, S::kColumns);
}

}  // namespace pe
