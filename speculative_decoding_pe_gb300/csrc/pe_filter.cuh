// Filtered distributions of logits rows: what pe_draft_sample and
// pe_verify_filtered share.
//
// A row's filter under (T, k, p, m): columns ordered by value, equal ones by
// column; kept are the first k; of those the smallest prefix that holds p of
// their weight; of those the ones of at least m of the largest weight.  Every
// step keeps a prefix of the order, so a cut is a value and, among the columns
// of that value, a last column (Cut below).
//
// A row lives in the shared memory of a cluster: one read of global memory,
// however often the cut's search looks at it.  Weights are
// w(x) = 2^((x - M) log2(e) / T), M the row's maximum, as a sum of two floats
// with some 32 bits: the draw falls between running sums of up to V weights, and
// with 24 bits a draw in a thousand of an unfiltered row would name the
// neighbour of the right column.  Where all columns count, the smallest weights, which hold little,
// are taken in fewer bits (small weights below).  Sums are exact integers or floats with
// what they drop, in a fixed order, so a call's results do not depend on timing.
#pragma once

#include "pe_cluster.cuh"
#include "pe_internal.cuh"
#include "pe_tma.cuh"

namespace pe {

constexpr int kFT = 256;          // threads of a filter CTA: four fit an SM
constexpr int kFW = kFT / 32;
constexpr int kListCap = 1024;    // columns of a candidate list
constexpr int kListK = 256;       // largest top-k whose columns the threads' maxima bound (one each)

// ------------------------------------------------------------------- weights
// 2^(j/32) as the sum of two floats.
__device__ const float2 kExp2Table[32] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f},
    {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f}, {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f},
    {0x1.172b840000000p+0f, -0x1.c157420000000p-27f}, {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f},
    {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}, {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f},
    {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f}, {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f},
    {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f}, {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f},
    {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f}, {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f},
    {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f}, {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f},
    {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f}, {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f},
    {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f}, {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f},
    {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f}, {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}, {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f},
    {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f}, {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f},
    {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f}, {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f},
    {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}, {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f},
};

// One row's scale: w(x) = 2^((x - M) c), c = log2(e) / T as two floats.  far: distance
// from M from which on a weight is nothing (2^-64).  A row with an infinity
// shares its weight among those columns.
struct Scale {
  float M, ch, cl, far, octave;  // octave: 1 / c
  bool inf;
};

// The parts of c and of min-p's floor that do not need the row.  64-bit arithmetic is
// slow on this GPU (a warp's instruction takes some 16 clocks): one thread of a CTA does it, while
// the row is on its way.
struct Rates {
  float ch, cl, far, octave;
  double log_m;  // T ln(m), where min-p is on
};
__device__ __forceinline__ Rates make_rates(float T, float m) {
  Rates r;
  const double t = T > 0.f ? (double)T : 1.0, c = 1.4426950408889634 / t;
  r.ch = __double2float_rz(c);
  r.cl = fmaxf((float)(c - (double)r.ch), 0x1p-120f);  // (above zero: -infinity times it is one)
  r.octave = (float)(t * 0.6931471805599453);
  r.far = 64.f * r.octave;
  r.log_m = m > 0.f && m < 1.f ? t * log((double)m) : 0.0;
  return r;
}
__device__ __forceinline__ Scale make_scale(float M, const Rates& r) {
  return Scale{M, r.ch, r.cl, r.far, r.octave, M == INFINITY};
}

// w(x) = hi + lo.  y = (x - M) c = n + j/32 + r with |r| <= 1/64;
// 2^y = 2^n 2^(j/32) (1 + q), q = 2^r - 1 from its Taylor series (the first
// term left out is below 2^-39).  The difference and the products are carried with
// their rounding errors; what is left is the rounding of q, 2^-31 at most.
__device__ __forceinline__ float2 weight(const Scale& s, const float2* table, float x) {
  if (s.inf) return make_float2(x == INFINITY ? 1.f : 0.f, 0.f);
  float d = x - s.M;
  const float bb = d - x;
  const float dl = (x - (d - bb)) - (s.M + bb);  // exact: d + dl = x - M
  const bool near = d > -s.far;  // not -inf, not NaN
  const float e0 = near ? dl : 0.f;
  d = near ? d : 0.f;
  const float p = d * s.ch;
  const float e = fmaf(d, s.ch, -p) + fmaf(d, s.cl, e0 * s.ch);
  const float z = p + 393216.f;  // 1.5 * 2^18: the sum's last bit is 1/32
  const int zi = __float_as_int(z) - 0x48c00000;
  const float r = (p - (z - 393216.f)) + e;
  const float2 t = table[zi & 31];
  const float in = fmaf(r, fmaf(r, fmaf(r, 0x1.3b2ab60000000p-7f, 0x1.c6b08e0000000p-5f), 0x1.ebfbe00000000p-3f), -0x1.05c6100000000p-29f);
  const float q = fmaf(r, 0x1.62e4300000000p-1f, r * in);
  const float two_n = near ? __int_as_float((127 + (zi >> 5)) << 23) : 0.f;
  return make_float2(t.x * two_n, fmaf(t.x, q, t.y) * two_n);
}

// Sum of weights: a float whose last bit is fixed by a bias larger than anything that
// is added (so that what an addition drops is exact), and the sum of what was dropped.
template <int kBias>
struct ShortSum {
  float s = (float)kBias, lo = 0.f;
  __device__ __forceinline__ void add(float h) {
    const float t = s + h;
    lo += h - (t - s);
    s = t;
  }
  // times 2^bits, as an integer: s - kBias is a multiple of the bias's last bit
  __device__ __forceinline__ unsigned long long fixed(int bits) const {
    const long long v = __float2ll_rn((s - (float)kBias) * __int_as_float((127 + bits) << 23)) +
                        __float2ll_rn(lo * __int_as_float((127 + bits) << 23));
    return v > 0 ? (unsigned long long)v : 0ull;
  }
};
// The same of weights as two floats, of any size and alike: what the first float drops goes to a
// second one with a bias of its own, of some 2^10 such pieces.  (In a plain sum, roundings of equal
// weights below half of the first one's last bit go one way: 1e-7 of them.)
template <int kBias>
struct WeightSum {
  static constexpr float kMid = (float)kBias / (1 << 13);
  float s = (float)kBias, mid = kMid, lo = 0.f;
  __device__ __forceinline__ void add(float h, float l) {
    const float w = h + l;  // (l may be a 64th of h: table value and rest)
    const float t = s + w, r = w - (t - s), u = mid + r;
    lo += (r - (u - mid)) + (l - (w - h));
    s = t;
    mid = u;
  }
  __device__ __forceinline__ bool positive() const { return (s - (float)kBias) + ((mid - kMid) + lo) > 0.f; }
  __device__ __forceinline__ unsigned long long fixed(int bits) const {
    const float up = __int_as_float((127 + bits) << 23);
    const long long v = __float2ll_rn((s - (float)kBias) * up) + __float2ll_rn((mid - kMid) * up) + __float2ll_rn(lo * up);
    return v > 0 ? (unsigned long long)v : 0ull;
  }
};
// One weight times 2^bits.
__device__ __forceinline__ unsigned long long fixed_weight(float2 w, int bits) {
  const float up = __int_as_float((127 + bits) << 23);
  const long long v = __float2ll_rn(w.x * up) + __float2ll_rn(w.y * up);
  return v > 0 ? (unsigned long long)v : 0ull;
}
// floor(u W) for u in [0,1)
__device__ __forceinline__ unsigned long long share_of(float u, unsigned long long W) {
  return __umul64hi(__float2ull_rz(u * 0x1p64f), W);
}
// w / W in fp32, W times 2^bits (off by half a step and 2^-31 of itself: the quotient's own rounding is
// corrected by the remainder).
__device__ __forceinline__ float ratio(float2 w, unsigned long long W, int bits) {
  const float up = __int_as_float((127 + bits) << 23);
  const float a = w.x * up, b = __ull2float_rz(W), bl = (float)(W - (unsigned long long)b);
  const float q = a / b;
  return q + (fmaf(-q, b, a) + (w.y * up - q * bl)) / b;
}
// The smallest whole number that is at least u W, and at least 1
__device__ __forceinline__ unsigned long long share_from(float u, unsigned long long W) {
  const unsigned long long f = __float2ull_rz(u * 0x1p64f);
  return max(__umul64hi(f, W) + (f * W != 0ull), 1ull);
}
constexpr int kSumBits = 44;   // row sums: up to 2^18 weights of at most 1
constexpr int kListBits = 52;  // list sums: up to 2^10

// Two sums, two products in one instruction each.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 a, a, b;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 a, a, b;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float exp2_hw(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Small weights: those of a vector whose largest is below 2^-16 of the row's, by the hardware's
// exponential of the exponent (x - M) c in 24 bits.  The part of c that 24 bits leave out would put all
// weights of a row off alike (5e-7 at T = 1.3) and is put in: c is split so that it is above zero, and a
// masked column's exponent stays -infinity.  fp32 rows also carry what the product's rounding drops, r:
// 2^(y + r) = 2^y (1 + r ln 2); a row's values may lie so close that the roundings go one way (2.7e-7 of the
// sum).  In bf16 rows they differ from value to value; carrying r there makes sums hardly better and takes
// 7 % longer (64 verifications under top-p).
// What is left of one weight: the difference's or the exponent's rounding and the exponential's own error
// (1.4e-7 at most), 2^-19 of itself in all (2^-18 below 2^-32).  Of a row's sum: the exponential's mean error,
// which is put back: -5.0e-8 to -5.4e-8 over fp32 values that fill an octave, -3.2e-8 to -7.9e-8 over the hundred
// different values of a bf16 row there (T from 0.3 to 2).
constexpr float kSmallMean = 5.1e-8f;  // of a small weight, to be added
constexpr float kNothing = -256.f;     // octaves, below what the exponential gives anything for

// Two of them, added to sum, and what their exponents lack, to rest (times ln 2).  clean: NaN may be there.
template <int DT>
__device__ __forceinline__ void add_small(const Scale& s, float2 x, bool clean, float2& sum, float2& rest) {
  const float2 rate = make_float2(s.ch, s.ch), rate_lo = make_float2(s.cl, s.cl);
  if (DT == PE_BF16 && clean) x = make_float2(fmaxf(x.x, -INFINITY), fmaxf(x.y, -INFINITY));
  float2 d = add2(x, make_float2(-s.M, -s.M));
  if (DT == PE_BF16) {
    const float2 y = fma2(d, rate, mul2(d, rate_lo));
    sum = add2(sum, make_float2(exp2_hw(y.x), exp2_hw(y.y)));
  } else {
    const float least = kNothing * s.octave;
    d = make_float2(fmaxf(d.x, least), fmaxf(d.y, least));  // (-infinity and NaN too)
    const float2 y = mul2(d, make_float2(-s.ch, -s.ch));    // (of the other sign)
    const float2 w = make_float2(exp2_hw(-y.x), exp2_hw(-y.y));
    sum = add2(sum, w);
    rest = fma2(w, fma2(d, rate_lo, fma2(d, rate, y)), rest);
  }
}
// One of them.
template <int DT>
__device__ __forceinline__ float small_weight(const Scale& s, float x) {
  float d = fmaxf(x, -INFINITY) - s.M;
  if (DT == PE_BF16) return exp2_hw(fmaf(d, s.ch, d * s.cl));
  d = fmaxf(d, kNothing * s.octave);
  const float y = d * s.ch, w = exp2_hw(y);
  return fmaf(w * 0.693147181f, fmaf(d, s.cl, fmaf(d, s.ch, -y)), w);
}

// ---------------------------------------------------------------- elements
template <int DT>
struct Elt;
template <>
struct Elt<PE_BF16> {
  static constexpr int kN = 8, kSize = 2, kKeyBits = 16;
  __device__ static __forceinline__ float get(uint4 q, int e) {
    const uint32_t w = (e >> 1) == 0 ? q.x : (e >> 1) == 1 ? q.y : (e >> 1) == 2 ? q.z : q.w;
    return (e & 1) ? bf16_hi(w) : bf16_lo(w);
  }
  // element e of vector i in shared memory
  __device__ static __forceinline__ float element(const uint4* v, int i, int e) {
    return __uint_as_float((uint32_t) reinterpret_cast<const unsigned short*>(v + i)[e] << 16);
  }
  // (a NaN gives way to the other operand)
  __device__ static __forceinline__ float max_of(uint4 q) {
    const uint32_t m = bf16x2_max(bf16x2_max(bf16x2_max(q.x, q.y), bf16x2_max(q.z, q.w)), 0xff80ff80u);
    return fmaxf(bf16_lo(m), bf16_hi(m));
  }
  __device__ static __forceinline__ float load(const char* row, int col) {
    return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(row) + col) << 16);
  }
};
template <>
struct Elt<PE_F32> {
  static constexpr int kN = 4, kSize = 4, kKeyBits = 32;
  __device__ static __forceinline__ float get(uint4 q, int e) {
    return __uint_as_float(e == 0 ? q.x : e == 1 ? q.y : e == 2 ? q.z : q.w);
  }
  __device__ static __forceinline__ float element(const uint4* v, int i, int e) {
    return reinterpret_cast<const float*>(v + i)[e];
  }
  __device__ static __forceinline__ float max_of(uint4 q) {
    return fmaxf(fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)),
                       fmaxf(__uint_as_float(q.z), __uint_as_float(q.w))), -INFINITY);
  }
  __device__ static __forceinline__ float load(const char* row, int col) {
    return __ldg(reinterpret_cast<const float*>(row) + col);
  }
};

// Order of values as unsigned integers; NaN as -infinity.
__device__ __forceinline__ uint32_t value_key(float x) { return ordered_bits(fmaxf(x, -INFINITY)); }
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// ---------------------------------------------------------------------- cuts
// Kept: x >= floor, and key(x) above `key`, or equal to it with col <= tie.
struct Cut {
  uint32_t key;
  int tie;
  float floor;
  __device__ __forceinline__ bool keeps(float x, int col) const {
    const uint32_t k = value_key(x);
    return x >= floor && (k > key || (k == key && col <= tie));
  }
};

// What is known of a row after its pass (verification).
struct RowCut {
  Cut cut;
  float M;
  float T;
  int listed;    // kept columns in the row's list, or -1 (not listed)
  int token;     // the draw from the row (bonus rows)
  double W;      // sum of kept weights; 0: nothing to keep; -1: bad parameters
  double wx;     // kept weight of the row's draft token; 0: not kept, or not in the vocabulary
};
struct Kept {  // a kept column and its weight times 2^kListBits
  unsigned long long w;
  int col;
  int pad;
};
constexpr int kKeptCap = 256;  // kept columns that a row's list holds

// Parameters of one request; false: not usable.
struct Asked {
  float T, p, m;
  int k;
};
struct AskedArrays {
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
};
__device__ __forceinline__ bool read_asked(const AskedArrays& a, int i, int V, Asked& o) {
  o.T = a.temperature ? __ldg(a.temperature + i) : 1.f;
  o.k = a.top_k ? __ldg(a.top_k + i) : 0;
  o.p = a.top_p ? __ldg(a.top_p + i) : 1.f;
  o.m = a.min_p ? __ldg(a.min_p + i) : 0.f;
  const bool ok = (o.T == 0.f || (o.T >= 0x1p-30f && o.T <= 0x1p30f)) && o.p == o.p && o.m == o.m;
  if (o.k <= 0 || o.k > V) o.k = V;
  if (o.T == 0.f) o.k = 1;
  return ok;
}
// Smallest value that min-p keeps (-infinity: all).
__device__ __forceinline__ float min_p_floor(const Asked& a, const Rates& r, float M) {
  if (!(a.m > 0.f) || a.T == 0.f) return -INFINITY;
  if (a.m >= 1.f || M == INFINITY) return M;
  return __double2float_ru((double)M + r.log_m);  // x >= t exactly when x >= this float
}

}  // namespace pe
