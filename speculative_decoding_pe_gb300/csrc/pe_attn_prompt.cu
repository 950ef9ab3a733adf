// Causal attention over whole packed prompts (pe_attn_prompt).
//
// One warp per row and query head, one pass over the keys with the running
// maximum and sum of the softmax; a lane holds D/32 elements.
#include "pe_attn.cuh"

namespace pe {

struct PromptParams {
  Segments seg;
  int Hq, Hkv;
  long long q_row, q_head, k_row, k_head, v_row, v_head;
  float scale_log2;
  const uint16_t *q, *k, *v;
  uint16_t* out;
  uint32_t* err;
};

template <int D>
__global__ void __launch_bounds__(kThreads) attn_prompt_kernel(const PromptParams p) {
  constexpr int E = D / 32;
  if (p.seg.offsets && !offsets_valid(p.seg.offsets, p.seg.B, p.seg.T, 0)) {
    if (threadIdx.x == 0) atomicOr(p.err, PE_ERR_OFFSETS);
    return;
  }
  const int lane = threadIdx.x & 31, G = p.Hq / p.Hkv;
  const long long nwarps = ((long long)gridDim.x * kThreads) >> 5;
  for (long long it = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
       it < (long long)p.seg.T * p.Hq; it += nwarps) {
    const int t = (int)(it / p.Hq), h = (int)(it - (long long)t * p.Hq), hk = h / G;
    const int first = p.seg.begin(p.seg.request(t));
    float q[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[e] = __uint_as_float((uint32_t)p.q[t * p.q_row + h * p.q_head + lane * E + e] << 16) *
             p.scale_log2;
      o[e] = 0.0f;
    }
    for (int j = first; j <= t; ++j) {
      const uint32_t* k = reinterpret_cast<const uint32_t*>(p.k + j * p.k_row + hk * p.k_head + lane * E);
      const uint32_t* v = reinterpret_cast<const uint32_t*>(p.v + j * p.v_row + hk * p.v_head + lane * E);
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < E / 2; ++e) s += q[2 * e] * bf16_lo(k[e]) + q[2 * e + 1] * bf16_hi(k[e]);
#pragma unroll
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
      l = l * f + w;
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        o[2 * e] = o[2 * e] * f + w * bf16_lo(v[e]);
        o[2 * e + 1] = o[2 * e + 1] * f + w * bf16_hi(v[e]);
      }
      m = mn;
    }
    const float r = 1.0f / l;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t*>(p.out + it * D + lane * E + e) = pack_bf16(o[e] * r, o[e + 1] * r);
  }
}

}  // namespace pe

extern "C" int pe_attn_prompt(const pe_attn_prompt_args* a, void* stream) {
  if (!a) return PE_EINVAL;
  if (int rc = pe_host::attn_sizes(a->T, a->B, a->Hq, a->Hkv, a->D, a->offsets, a->scale)) return rc;
  const int64_t strides[] = {a->q_row, a->q_head, a->k_row, a->k_head, a->v_row, a->v_head};
  for (int64_t s : strides)
    if (s < 0 || s > INT32_MAX) return PE_EINVAL;
  if (a->T == 0) return PE_OK;
  if (!a->q || !a->k || !a->v || !a->out || !a->workspace || !a->err) return PE_EINVAL;
  if (!pe_host::aligned16(a->q) || !pe_host::aligned16(a->k) || !pe_host::aligned16(a->v) ||
      !pe_host::aligned16(a->out) || !pe_host::aligned16(a->workspace))
    return PE_EALIGN;
  for (int64_t s : strides)
    if (s % 8) return PE_EALIGN;
  pe_host::DeviceInfo dev;
  if (pe_host::device_info(&dev) != PE_OK) return PE_ECUDA;
  pe::PromptParams p;
  p.seg = {a->offsets, a->T, a->B};
  p.Hq = a->Hq, p.Hkv = a->Hkv;
  p.q_row = a->q_row, p.q_head = a->q_head, p.k_row = a->k_row, p.k_head = a->k_head;
  p.v_row = a->v_row, p.v_head = a->v_head;
  p.scale_log2 = a->scale * 1.4426950408889634f;
  p.q = static_cast<const uint16_t*>(a->q);
  p.k = static_cast<const uint16_t*>(a->k);
  p.v = static_cast<const uint16_t*>(a->v);
  p.out = static_cast<uint16_t*>(a->out);
  p.err = a->err;
  const int grid = dev.sm_count * 8;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->D == 64)
    pe::attn_prompt_kernel<64><<<grid, pe::kThreads, 0, s>>>(p);
  else
    pe::attn_prompt_kernel<128><<<grid, pe::kThreads, 0, s>>>(p);
  return pe_host::launch_status();
}
