// Thread-block clusters: rank, barrier, addresses in another CTA's shared memory.
#pragma once

#include <atomic>

#include <cuda_runtime.h>
#include <stdint.h>

namespace pe {

constexpr int kMaxCluster = 16;  // (above 8: kernels that allow a non-portable size)

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Barriers whose lanes arrive one by one (no .aligned).  The forms for whole warps count
// a warp as soon as some of its lanes come by: in the list's code, where lanes of a warp
// differ in how many columns they hold from one barrier to the next, the compiled warp
// reached __syncthreads() in two parts, and the barrier let the others go too early.
__device__ __forceinline__ void cta_sync() { asm volatile("barrier.cta.sync 0;" ::: "memory"); }
// The same, and how many threads have `yes`.
__device__ __forceinline__ int cta_count(bool yes) {
  int n;
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.popc.u32 %0, 0, p;\n\t}"
               : "=r"(n)
               : "r"((uint32_t)yes)
               : "memory");
  return n;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// The same variable in the shared memory of the cluster's CTA `rank`.
template <class T>
__device__ __forceinline__ T* at_rank(T* p, uint32_t rank) {
  T* q;
  asm("mapa.u64 %0, %1, %2;" : "=l"(q) : "l"(p), "r"(rank));
  return q;
}

}  // namespace pe

namespace pe_host {

// Clusters of more than eight CTAs must be opted into once per kernel and device.
template <class K>
bool allow_wide_clusters(K kernel, std::atomic<unsigned long long>& done_mask) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  const unsigned long long bit = 1ull << dev;
  if (done_mask.load(std::memory_order_relaxed) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) return false;
  done_mask.fetch_or(bit);
  return true;
}

// A launch in clusters of C CTAs; `dependent`: the kernel may start before the one
// ahead of it on the stream has finished, and waits for it (griddepcontrol.wait).
template <class K, class P>
cudaError_t launch_clusters(K kernel, dim3 grid, int threads, int C, size_t smem, bool dependent, cudaStream_t st,
                            const P& p) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace pe_host
