// Causal attention over whole packed prompts (pe_attn_prompt): the tensor-core
// attention of pe_attn_mma.cuh with queries, keys and values brought by TMA.
//
// A query tile is the G heads of a key head times 128/G tokens, one 3-axis box;
// a key tile 128 tokens of one head.  Tiles may reach past a prompt's end into
// the next prompt, or past the last row (filled with zeros): their scores are
// masked, and their values must not meet even a weight of zero, because zero
// times an infinity is a NaN.  So a warp looks over the value tiles that any
// row masks: rows past the prompt are cleared, and elements that are not finite
// are taken out and given back at the end to the rows that see them.
//
// Measured (in a graph): two prompts of 18 000 tokens, 32 heads of 128 on 4: 3.46 ms,
// 1.49 PFLOP/s of the causal half, 78 % of a library product's burst rate (3.65 ms in a
// long run under the power cap, 81 % of its sustained rate): bound by the products.
// Eight prompts of 4600 tokens, 64 heads of 64 on 8: 2.06 ms, 0.88 PFLOP/s: bound by the
// softmax, whose exponentials alone take 0.72 ms and its other instructions about as
// much.  Sixteen prompts of up to 131 tokens: 17.8 us, a chain of a plan, two or three
// tiles a CTA, and their stores.
#include "pe_attn_mma.cuh"

namespace pe {

struct PromptParams {
  Segments seg;
  int Hkv, G;
  SoftmaxArgs softmax;
};

constexpr int kPromptThreads = 12 * 32;

// Query, key and value tiles into shared memory; one thread.
template <int D, class Control>
__device__ void bring_tiles(const Line<false>& line, Control& c, uint8_t* smem, const CUtensorMap* qm,
                            const CUtensorMap* km, const CUtensorMap* vm) {
  using S = AttnShape<D, false>;
  volatile int* dead = &c.dead;
  Walk w = c.start;
  uint32_t k = 0, nq[2] = {0, 0};
  const uint32_t q_bytes = line.G * line.span * D * 2;
  while (walk_next(line, w)) {
    for (int s = 0; s < 2; ++s) {
      if (!visits(line, w, s).count) continue;
      if (!wait_or_dead(&c.q_empty[s], (nq[s]++ & 1) ^ 1, dead)) return;
      mbar_arrive_expect_tx(&c.q_full[s], q_bytes);
      for (int x = 0; x < D / 64; ++x)
        tma_load_3d(smem + S::kQ + s * S::kOperand + x * kTile * 128, qm, 64 * x, w.h * line.G,
                    w.first + (2 * w.mt + s) * line.span, &c.q_full[s]);
    }
    for (int j = w.t0; j < w.t1; ++j, ++k) {
      const uint32_t st = k % S::kStages, phase = (k / S::kStages) & 1;
      const int row = w.first + j * kTile;
      if (!wait_or_dead(&c.k_empty[st], phase ^ 1, dead)) return;
      mbar_arrive_expect_tx(&c.k_full[st], S::kOperand);
      for (int x = 0; x < D / 64; ++x)
        tma_load_3d(smem + S::kK + st * S::kOperand + x * kTile * 128, km, 64 * x, w.h, row, &c.k_full[st]);
      if (!wait_or_dead(&c.v_empty[st], phase ^ 1, dead)) return;
      mbar_arrive_expect_tx(&c.v_full[st], S::kOperand);
      for (int x = 0; x < D / 64; ++x)
        tma_load_3d(smem + S::kV + st * S::kOperand + x * kTile * 128, vm, 64 * x, w.h, row, &c.v_full[st]);
    }
  }
}

// 0 x + sum for two bf16.
__device__ __forceinline__ uint32_t zero_times(uint32_t x, uint32_t sum) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(x), "r"(0u), "r"(sum));
  return d;
}

// Values on their way to the tensor core; one warp.
template <int D, class Control>
__device__ void look_over_values(const Line<false>& line, Control& c, uint8_t* smem) {
  using S = AttnShape<D, false>;
  volatile int* dead = &c.dead;
  const int lane = threadIdx.x & 31;
  Walk w = c.start;
  uint32_t k = 0;
  for (int segment = 0; walk_next(line, w); ++segment) {
    const int least = 2 * w.mt * line.span + 1;  // keys that the item's first row sees
    uint32_t any = 0;
    if (lane == 0) c.any_not_finite[segment % kNotes] = 0;
    for (int j = w.t0; j < w.t1; ++j, ++k) {
      const uint32_t st = k % S::kStages;
      if (!wait_warp(&c.v_full[st], (k / S::kStages) & 1, dead)) return;
      if ((j + 1) * kTile > least) {
        uint8_t* tile = smem + S::kV + st * S::kOperand;
#pragma unroll 1
        for (int word = 0; word < 4; ++word) {
          const int row = word * 32 + lane, key = j * kTile + row;
          // the lanes take a row's pieces in different orders (banks)
          auto piece = [&](int x, int i) {
            return reinterpret_cast<uint4*>(tile + x * kTile * 128 + row * 128) + ((i + lane) & 7);
          };
          bool found = false;
          if (key >= w.rows) {
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
#pragma unroll
              for (int i = 0; i < 8; ++i) *piece(x, i) = make_uint4(0, 0, 0, 0);
          } else if (key >= least) {
            uint32_t sum[4] = {0, 0, 0, 0};  // zero times the elements: a NaN if one is not finite
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint4 y = *piece(x, i);
                sum[0] = zero_times(y.x, sum[0]), sum[1] = zero_times(y.y, sum[1]);
                sum[2] = zero_times(y.z, sum[2]), sum[3] = zero_times(y.w, sum[3]);
              }
            found = ((sum[0] | sum[1] | sum[2] | sum[3]) & 0x7fff7fffu) != 0;
            if (found)
#pragma unroll 1
              for (int i = 0; i < D / 8; ++i) {
                uint32_t* y = reinterpret_cast<uint32_t*>(piece(i / 8, i % 8));
                for (int e = 0; e < 4; ++e) {
                  if ((y[e] & 0x7f80u) == 0x7f80u) y[e] &= 0xffff0000u;
                  if ((y[e] & 0x7f800000u) == 0x7f800000u) y[e] &= 0xffffu;
                }
              }
          }
          const uint32_t bits = __ballot_sync(0xffffffffu, found);
          any |= bits;
          if (lane == 0) {
            c.not_finite[segment % kNotes][(j - least / kTile) * 4 + word] = bits;
            c.any_not_finite[segment % kNotes] = any != 0;
          }
        }
        fence_async_shared();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.v_ready[st]);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kPromptThreads, 1)
    attn_prompt_kernel(const PromptParams p, const __grid_constant__ CUtensorMap qm,
                       const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm) {
  using S = AttnShape<D, false>;
  extern __shared__ uint8_t raw[];
  __shared__ AttnControl<S::kStages> c;
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  long long* prefix = reinterpret_cast<long long*>(smem + S::kData);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) c.init(1, 1, 1);
  Line<false> line{p.seg, p.Hkv, p.G, kTile / p.G, nullptr, nullptr};
  if (!plan(line, 2, 2, c, prefix, nullptr, reinterpret_cast<long long*>(smem), nullptr, nullptr, 0, p.softmax.err)) return;
  if (c.start.u >= c.start.end) return;  // fewer parts than CTAs
  if (warp == 8) tmem_alloc(&c.tmem, S::kColumns);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // 12 warps of 168 registers: 200 for the softmax's rows, 104 for the others
  if (warp < 8)
    take_registers<200>();
  else
    give_registers<104>();
  if (warp < 8) {
    softmax_rows<D, false>(line, c, p.softmax, warp >> 2);
  } else if (warp == 8) {
    if (elect_one()) issue_products<D, false>(line, c, smem_addr(smem));
  } else if (warp == 9) {
    if (elect_one()) bring_tiles<D>(line, c, smem, &qm, &km, &vm);
  } else if (warp == 10) {
    look_over_values<D>(line, c, smem);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (c.dead) leave_after_timeout<D, false>(c, p.softmax.err);
  if (warp == 8) tmem_dealloc(c.tmem, S::kColumns);
}

}  // namespace pe

namespace {

// Rows [T, heads, D] as a 3-axis map with boxes of 64 elements x heads x tokens.
bool encode_rows(CUtensorMap* map, const void* base, int D, int heads, int T, int64_t head, int64_t row,
                 int box_heads, int box_rows) {
  using Encode = decltype(&cuTensorMapEncodeTiled);
  static std::atomic<Encode> cached{nullptr};
  Encode encode = cached.load(std::memory_order_relaxed);
  if (!encode) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return false;
    encode = reinterpret_cast<Encode>(f);
    cached.store(encode, std::memory_order_relaxed);
  }
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T};
  // the stride of an axis of one element is never used
  const cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? head : D) * 2, (cuuint64_t)(T > 1 ? row : D) * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  const cuuint32_t steps[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
int launch(const pe_attn_prompt_args* a, const pe::PromptParams& p, int sms, cudaStream_t s) {
  CUtensorMap q, k, v;
  if (!encode_rows(&q, a->q, D, a->Hq, a->T, a->q_head, a->q_row, p.G, pe::kTile / p.G) ||
      !encode_rows(&k, a->k, D, a->Hkv, a->T, a->k_head, a->k_row, 1, pe::kTile) ||
      !encode_rows(&v, a->v, D, a->Hkv, a->T, a->v_head, a->v_row, 1, pe::kTile))
    return PE_ECUDA;
  static std::atomic<unsigned long long> allowed{0};
  const int most = pe::AttnShape<D, false>::kData + 1024 + 8 * (PE_MAX_ATTN_B + 1);
  if (!pe_host::allow_smem(pe::attn_prompt_kernel<D>, most, allowed)) return PE_ECUDA;
  const int bytes = pe::AttnShape<D, false>::kData + 1024 + 8 * (a->B + 1);
  const int grid = sms < pe::kAttnCtas ? sms : pe::kAttnCtas;
  pe::attn_prompt_kernel<D><<<grid, pe::kPromptThreads, bytes, s>>>(p, q, k, v);
  return pe_host::launch_status();
}

}  // namespace

extern "C" int pe_attn_prompt(const pe_attn_prompt_args* a, void* stream) {
  if (!a) return PE_EINVAL;
  if (int rc = pe_host::attn_sizes(a->T, a->B, a->Hq, a->Hkv, a->D, a->offsets, a->scale)) return rc;
  const int64_t strides[][2] = {{a->q_row, a->T}, {a->q_head, a->Hq}, {a->k_row, a->T},
                                {a->k_head, a->Hkv}, {a->v_row, a->T}, {a->v_head, a->Hkv}};
  for (auto& s : strides)
    if (s[0] < 0 || s[0] > INT32_MAX || (s[0] == 0 && s[1] > 1)) return PE_EINVAL;
  if (a->T == 0) return PE_OK;
  if (!a->q || !a->k || !a->v || !a->out || !a->workspace || !a->err) return PE_EINVAL;
  if (!pe_host::aligned16(a->q) || !pe_host::aligned16(a->k) || !pe_host::aligned16(a->v) ||
      !pe_host::aligned16(a->out) || !pe_host::aligned16(a->workspace))
    return PE_EALIGN;
  for (auto& s : strides)
    if (s[0] % 8) return PE_EALIGN;
  pe_host::DeviceInfo dev;
  if (pe_host::device_info(&dev) != PE_OK) return PE_ECUDA;
  pe::PromptParams p;
  p.seg = {a->offsets, a->T, a->B};
  p.Hkv = a->Hkv, p.G = a->Hq / a->Hkv;
  p.softmax.Hq = a->Hq;
  p.softmax.table_keys = 0;
  p.softmax.scale_log2 = a->scale * 1.4426950408889634f;
  p.softmax.positions = nullptr;
  p.softmax.is_rejected = nullptr;
  p.softmax.v = static_cast<const uint16_t*>(a->v);
  p.softmax.v_row = a->v_row, p.softmax.v_head = a->v_head;
  p.softmax.out = static_cast<uint16_t*>(a->out);
  p.softmax.ws = static_cast<uint8_t*>(a->workspace);
  p.softmax.err = a->err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a->D == 64 ? launch<64>(a, p, dev.sm_count, s) : launch<128>(a, p, dev.sm_count, s);
}
