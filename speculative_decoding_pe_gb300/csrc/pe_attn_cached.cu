// Attention over the 4-bit paged KV cache (pe_attn_cached).
//
// One warp per row and query head, one pass over the keys with the running
// maximum and sum of the softmax; a lane holds D/32 elements.
#include "pe_attn_few.cuh"

namespace pe {

template <int D>
__global__ void __launch_bounds__(kThreads) attn_cached_kernel(const CachedParams p) {
  using R = Record<D>;
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
    const int b = p.seg.request(t);
    bool bad = false;
    const int limit = row_limit(p.positions, p.is_rejected, t, p.table_keys, bad);
    if (bad && lane == 0) atomicOr(p.err, PE_ERR_BLOCK_RANGE);
    float q[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[e] = __uint_as_float((uint32_t)p.q[it * D + lane * E + e] << 16) * p.scale_log2;
      o[e] = 0.0f;
    }
    for (int j = 0; j < limit; ++j) {
      const int blk = __ldg(p.block_table + (long long)b * p.bt_width + j / p.block_size);
      if (blk < 0 || blk >= p.num_blocks) {
        if (lane == 0) atomicOr(p.err, PE_ERR_BLOCK_RANGE);
        continue;
      }
      const uint8_t* rec = p.cache + record_offset((long long)blk * p.block_size + j % p.block_size,
                                                   p.block_size, p.Hkv, hk, R::kBytes);
      const int row = j & 15, x = lane * E;
      float k[8], v[8], ks, vs, unused;
      f16x2_to_f32(e4m3_f16x2(rec[R::kKs + row * R::kScaleRow + x / 16]), ks, unused);
      f16x2_to_f32(e4m3_f16x2(rec[R::kVs + row * R::kScaleRow + x / 16]), vs, unused);
      uint32_t kw[4], vw[4];
      e2m1x8_f16(E == 2 ? rec[R::kK + row * R::kRow + x / 2]
                        : *reinterpret_cast<const uint16_t*>(rec + R::kK + row * R::kRow + x / 2), kw);
      e2m1x8_f16(E == 2 ? rec[R::kV + row * R::kRow + x / 2]
                        : *reinterpret_cast<const uint16_t*>(rec + R::kV + row * R::kRow + x / 2), vw);
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        f16x2_to_f32(kw[e / 2], k[e], k[e + 1]);
        f16x2_to_f32(vw[e / 2], v[e], v[e + 1]);
        s += q[e] * (k[e] * ks) + q[e + 1] * (k[e + 1] * ks);
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
      l = l * f + w;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * f + w * (v[e] * vs);
      m = mn;
    }
    const float r = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t*>(p.out + it * D + lane * E + e) = pack_bf16(o[e] * r, o[e + 1] * r);
  }
}

}  // namespace pe

namespace {

template <int D, int NB>
int launch_few(const pe::CachedParams& p, int sms, cudaStream_t s) {
  static std::atomic<unsigned long long> allowed{0};
  const int most = pe::FewShape<D>::kBytes + 12 * (PE_MAX_ATTN_B + 1);
  if (!pe_host::allow_smem(pe::attn_few_kernel<D, NB>, most, allowed)) return PE_ECUDA;
  const int bytes = pe::FewShape<D>::kBytes + 12 * (p.seg.B + 1);
  const int grid = 2 * (sms < pe::kAttnCtas ? sms : pe::kAttnCtas);
  pe::attn_few_kernel<D, NB><<<grid, 256, bytes, s>>>(p);
  return pe_host::launch_status();
}

}  // namespace

extern "C" size_t pe_workspace_bytes_attn(int32_t D) {
  return D == 64 || D == 128 ? pe::AttnWorkspace::bytes(D) : 0;
}

extern "C" int pe_attn_cached(const pe_attn_cached_args* a, void* stream) {
  if (!a) return PE_EINVAL;
  if (int rc = pe_host::attn_sizes(a->T, a->B, a->Hq, a->Hkv, a->D, a->offsets, a->scale)) return rc;
  if (a->block_size < 16 || a->block_size % 16 || a->bt_width < 1 ||
      (int64_t)a->bt_width * a->block_size > INT32_MAX - 256 || a->num_blocks < 1 ||
      a->num_blocks > (INT64_MAX >> 8) / ((int64_t)a->Hkv * a->block_size * a->D))
    return PE_EINVAL;
  if (a->T == 0) return PE_OK;
  if (!a->q || !a->cache || !a->block_table || !a->positions || !a->out || !a->workspace || !a->err)
    return PE_EINVAL;
  if (!pe_host::aligned16(a->q) || !pe_host::aligned16(a->cache) || !pe_host::aligned16(a->out) ||
      !pe_host::aligned16(a->workspace))
    return PE_EALIGN;
  pe_host::DeviceInfo dev;
  if (pe_host::device_info(&dev) != PE_OK) return PE_ECUDA;
  pe::CachedParams p;
  p.seg = {a->offsets, a->T, a->B};
  p.Hq = a->Hq, p.Hkv = a->Hkv, p.block_size = a->block_size, p.bt_width = a->bt_width;
  p.table_keys = a->bt_width * a->block_size;
  p.num_blocks = a->num_blocks;
  p.scale_log2 = a->scale * 1.4426950408889634f;
  p.q = static_cast<const uint16_t*>(a->q);
  p.cache = static_cast<const uint8_t*>(a->cache);
  p.block_table = a->block_table;
  p.positions = a->positions;
  p.is_rejected = a->is_rejected;
  p.out = static_cast<uint16_t*>(a->out);
  p.err = a->err;
  p.ws = static_cast<uint8_t*>(a->workspace);
  const int grid = dev.sm_count * 8;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t rows = a->offsets ? INT64_MAX : (int64_t)(a->T / a->B) * (a->Hq / a->Hkv);
  if (rows <= 8) return a->D == 64 ? launch_few<64, 1>(p, dev.sm_count, s) : launch_few<128, 1>(p, dev.sm_count, s);
  if (rows <= 16) return a->D == 64 ? launch_few<64, 2>(p, dev.sm_count, s) : launch_few<128, 2>(p, dev.sm_count, s);
  if (a->D == 64)
    pe::attn_cached_kernel<64><<<grid, pe::kThreads, 0, s>>>(p);
  else
    pe::attn_cached_kernel<128><<<grid, pe::kThreads, 0, s>>>(p);
  return pe_host::launch_status();
}
