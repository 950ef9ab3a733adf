// What the attention kernels share: segments, workspace, argument checks.
#pragma once

#include <math.h>

#include "pe_internal.cuh"
#include "pe_kv.cuh"

namespace pe {

// Segment b of the packed rows: offsets[b..b+1], or T/B rows each.
struct Segments {
  const int32_t* offsets;
  int T, B;
  __device__ int begin(int b) const { return offsets ? __ldg(offsets + b) : b * (T / B); }
  __device__ int end(int b) const { return offsets ? __ldg(offsets + b + 1) : (b + 1) * (T / B); }
};

// Keys that a row of the cached attention sees.
__device__ __forceinline__ int row_limit(const int32_t* positions, const uint8_t* is_rejected,
                                         int t, int table_keys, bool& bad) {
  const int gone = is_rejected ? __ldg(is_rejected + t) : 0, pos = __ldg(positions + t);  // (both loads at once)
  if (gone) return 0;
  if (pos < 0) {
    bad = true;
    return 0;
  }
  if (pos >= table_keys) {
    bad = true;
    return table_keys;
  }
  return pos + 1;
}

// The call over the cache.
struct CachedParams {
  Segments seg;
  int Hq, Hkv, block_size, bt_width, table_keys;
  long long num_blocks;
  float scale_log2;
  const uint16_t* q;
  const uint8_t* cache;
  const int32_t* block_table;
  const int32_t* positions;
  const uint8_t* is_rejected;
  uint16_t* out;
  uint8_t* ws;
  uint32_t* err;
  int together;  // the CTAs run at once and add up cut items together
};

// The power of two to take out of a row whose largest magnitude is `most`, as
// (factor, its inverse); the exponents stay those of normal numbers.
__device__ __forceinline__ float2 row_factor(float most) {
  uint32_t e = __float_as_uint(most) >> 23;
  if (most == 0.0f || e >= 255) return make_float2(1.0f, 1.0f);
  e = min(max(e, 1u), 252u);
  return make_float2(__uint_as_float((254 - e) << 23), __uint_as_float(e << 23));
}

// Scratch: one counter per CTA that begins a split item, then three partial
// results per CTA of up to 256 rows (fp32 sums, maximum and total of a row).
constexpr int kAttnCtas = 152;
struct AttnWorkspace {
  static constexpr size_t kPartials = 4096;  // byte offset; counters before it
  __host__ __device__ static constexpr size_t partial_bytes(int D) { return (size_t)256 * (D + 2) * 4; }
  __host__ __device__ static constexpr size_t bytes(int D) { return kPartials + 3 * kAttnCtas * partial_bytes(D); }
};

}  // namespace pe

namespace pe_host {

// The checks that both attention calls share (sizes only).
inline int attn_sizes(int T, int B, int Hq, int Hkv, int D, const void* offsets, float scale) {
  if (T < 0 || B < 1 || B > PE_MAX_ATTN_B || Hq < 1 || Hkv < 1 || Hq % Hkv ||
      Hq / Hkv > PE_MAX_ATTN_G || (D != 64 && D != 128) || !isfinite(scale) || !(scale > 0.0f))
    return PE_EINVAL;
  if (!offsets && T % B) return PE_EINVAL;
  if (T > ((int64_t)1 << 40) / ((int64_t)Hq * D)) return PE_EINVAL;
  return PE_OK;
}

}  // namespace pe_host
