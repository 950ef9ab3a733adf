// Attention over the 4-bit paged KV cache (pe_attn_cached): which kernel takes it.
#include "pe_attn_few.cuh"
#include "pe_attn_many.cuh"

namespace {

// May items have so many parts (of 256 keys at least) that their CTAs add them up
// together?  A cooperative launch costs 1.3 us.  (Items: at most those of B requests
// that fill their last one by a token.)
bool cut_often(const pe::CachedParams& p, int grid) {
  const int64_t span = pe::kTile / (p.Hq / p.Hkv);
  return p.table_keys >= pe::kTogether * 256 && 2 * (int64_t)p.Hkv * (p.seg.B + p.seg.T / span) <= grid;
}

// Together: cooperative, so that every CTA runs at once.  A refusal (other work
// holds part of the GPU) leaves no error behind.
template <class Kernel>
int launch(Kernel* kernel, int grid, int threads, int bytes, pe::CachedParams p, cudaStream_t s) {
  p.together = cut_often(p, grid);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeCooperative;
  attr.val.cooperative = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = p.together ? 1 : 0;
  if (p.together && cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
    (void)cudaGetLastError();
    p.together = cfg.numAttrs = 0;
  }
  if (!p.together) (void)cudaLaunchKernelEx(&cfg, kernel, p);
  return pe_host::launch_status();
}

template <int D, int NB>
int launch_few(const pe::CachedParams& p, int sms, cudaStream_t s) {
  static std::atomic<unsigned long long> allowed{0};
  const int most = pe::FewShape<D>::kBytes + 12 * (PE_MAX_ATTN_B + 1);
  if (!pe_host::allow_smem(pe::attn_few_kernel<D, NB>, most, allowed)) return PE_ECUDA;
  const int bytes = pe::FewShape<D>::kBytes + 12 * (p.seg.B + 1);
  const int grid = 2 * (sms < pe::kAttnCtas ? sms : pe::kAttnCtas);
  return launch(pe::attn_few_kernel<D, NB>, grid, 256, bytes, p, s);
}

template <int D>
int launch_many(const pe::CachedParams& p, int sms, cudaStream_t s) {
  static std::atomic<unsigned long long> allowed{0};
  constexpr int kData = pe::AttnShape<D, true>::kData + 1024;
  if (!pe_host::allow_smem(pe::attn_many_kernel<D>, kData + 12 * (PE_MAX_ATTN_B + 1), allowed)) return PE_ECUDA;
  const int grid = sms < pe::kAttnCtas ? sms : pe::kAttnCtas;
  return launch(pe::attn_many_kernel<D>, grid, pe::kManyThreads, kData + 12 * (p.seg.B + 1), p, s);
}

}  // namespace

extern "C" size_t pe_workspace_bytes_attn(int32_t D) {
  return D == 64 || D == 128 ? pe::AttnWorkspace::bytes(D) : 0;
}

extern "C" int pe_attn_cached(const pe_attn_cached_args* a, void* stream) {
  if (!a) return PE_EINVAL;
  if (int rc = pe_host::attn_sizes(a->T, a->B, a->Hq, a->Hkv, a->D, a->offsets, a->scale)) return rc;
  if (!pe_host::cache_sizes_ok(a->num_blocks, a->block_size, a->Hkv, a->D) || a->bt_width < 1 ||
      (int64_t)a->bt_width * a->block_size > INT32_MAX - 256)
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // Rows of a request that are known to be few: 64 requests of 8000 keys, in a graph, 8
  // rows 96 us in the few-row kernel against 190 in the other, 16 rows 145 against 190 (8
  // heads of 64); 86 against 161 and 150 against 161 (4 heads of 128).  With offsets they
  // are not known here.
  const int64_t rows = a->offsets ? INT64_MAX : (int64_t)(a->T / a->B) * (a->Hq / a->Hkv);
  if (rows <= 8) return a->D == 64 ? launch_few<64, 1>(p, dev.sm_count, s) : launch_few<128, 1>(p, dev.sm_count, s);
  if (rows <= 16) return a->D == 64 ? launch_few<64, 2>(p, dev.sm_count, s) : launch_few<128, 2>(p, dev.sm_count, s);
  return a->D == 64 ? launch_many<64>(p, dev.sm_count, s) : launch_many<128>(p, dev.sm_count, s);
}
