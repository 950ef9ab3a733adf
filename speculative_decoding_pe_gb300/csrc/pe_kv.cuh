// The 4-bit paged KV cache: record layout and conversions.
//
// A record holds 16 tokens of one (block, head): key codes [16][D/2], value
// codes [16][D/2], key scales [16][D/16], value scales [16][D/16], 18*D bytes
// in all.  One record is one contiguous run of 1152 (D = 64) or 2304 bytes, a
// multiple of 128, so that a reader of the attention fetches keys, values and
// scales of 16 tokens with one bulk copy whatever the page size is.
#pragma once

#include "pe_internal.cuh"

namespace pe {

constexpr int kRecTokens = 16;

template <int D>
struct Record {
  static constexpr int kRow = D / 2;         // code bytes of a token
  static constexpr int kScaleRow = D / 16;   // scale bytes of a token
  static constexpr int kK = 0;
  static constexpr int kV = 16 * kRow;
  static constexpr int kKs = 32 * kRow;
  static constexpr int kVs = kKs + 16 * kScaleRow;
  static constexpr int kBytes = 18 * D;
};

// Byte offset of the record of token `slot` (a slot of the whole cache) and head h.
__device__ __forceinline__ long long record_offset(long long slot, int block_size, int Hkv,
                                                   int h, int rec_bytes) {
  // (a 64-bit division takes some hundred instructions)
  const long long block =
      (slot >> 32) == 0 ? (long long)((uint32_t)slot / (uint32_t)block_size) : slot / block_size;
  const int sub = (int)(slot - block * block_size) >> 4;
  return ((block * Hkv + h) * (block_size >> 4) + sub) * rec_bytes;
}

// Two floats as bf16, `lo` in the low half (to nearest, ties to even).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// e4m3 byte of x >= 0 (to nearest, ties to even, saturating at 448).
__device__ __forceinline__ uint32_t to_e4m3(float x) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.0f), "f"(x));
  return d & 0xffu;
}

// Two scale bytes as f16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)two));
  return d;
}
// The scale byte `b` in both halves, as f16.
__device__ __forceinline__ uint32_t e4m3_f16x2(uint32_t b) { return e4m3x2_f16x2(b | (b << 8)); }

// Four bytes of codes as eight f16 numbers (exact): d[i] holds elements 2i, 2i+1.
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&d)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(w));
}

// Eight floats as e2m1 codes in four bytes (to nearest, ties to even, saturating).
__device__ __forceinline__ uint32_t to_e2m1x8(const float* x) {
  uint32_t d;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(d)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return d;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Products of two f16 pairs as fp32 (exact).
__device__ __forceinline__ void mul_f16x2_f32(uint32_t x, uint32_t y, float& lo, float& hi) {
  asm("{\n\t.reg .f16 a, b, c, d;\n\tmov.b32 {a, b}, %2;\n\tmov.b32 {c, d}, %3;\n\t"
      "fma.rn.f32.f16 %0, a, c, %4;\n\tfma.rn.f32.f16 %1, b, d, %4;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(x), "r"(y), "f"(0.0f));
}
// The same with one half of y for both.
template <bool kHigh>
__device__ __forceinline__ void mul_f16x2_f32_by(uint32_t x, uint32_t y, float& lo, float& hi) {
  asm("{\n\t.reg .f16 a, b, c, d, f;\n\tmov.b32 {a, b}, %2;\n\tmov.b32 {c, d}, %3;\n\t"
      ".reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\tselp.b16 f, d, c, p;\n\t"
      "fma.rn.f32.f16 %0, a, f, %4;\n\tfma.rn.f32.f16 %1, b, f, %4;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(x), "r"(y), "f"(0.0f), "n"(kHigh));
}

__device__ __forceinline__ void f16x2_to_f32(uint32_t w, float& lo, float& hi) {
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(w));
}

}  // namespace pe

namespace pe_host {

// The sizes of a cache.  One division after another: the product of the divisors may
// pass 64 bits, and be zero.
inline bool cache_sizes_ok(int64_t num_blocks, int32_t block_size, int32_t Hkv, int32_t D) {
  return Hkv >= 1 && (D == 64 || D == 128) && block_size >= 16 && block_size % 16 == 0 && num_blocks >= 1 &&
         num_blocks <= (INT64_MAX >> 8) / Hkv / block_size / D;
}

}  // namespace pe_host
