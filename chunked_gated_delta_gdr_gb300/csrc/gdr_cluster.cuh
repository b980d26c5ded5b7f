// gdr_cluster.cuh -- thread-block clusters: ranks, barriers, addresses in other blocks' shared memory, launches.
#pragma once

#include "gdr_mix.cuh"
#include "gdr_tc.cuh"

namespace gdr {
namespace mix {
namespace {

constexpr int kMostCl = 16;  // blocks of a cluster (over 8 with the device's consent)

__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
__device__ __forceinline__ int cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return (int)r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// No block ends while another may write to it.
__device__ __forceinline__ void cluster_leave() {
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  cluster_wait();
}
__device__ __forceinline__ uint32_t at_rank(const void *p, int rank) {
  uint32_t to;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(tc::smem_u32(p)), "r"(rank));
  return to;
}

template <typename... P, typename... A>
cudaError_t launch_clusters(void (*kernel)(P...), int blocks, int cluster, int threads,
                            int smem, cudaStream_t stream, A... args) {
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)blocks);
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = (size_t)smem;
  c.stream = stream;
  c.attrs = at;
  c.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

// Clusters of `cl` blocks that run at once (asked for once for each device and size; -1: unknown).
template <typename K>
int clusters_at_once(K *kernel, int cl, int threads, int smem,
                     std::atomic<int> (&known)[64][kMostCl + 1]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  if (dev >= 0 && dev < 64) {
    const int n = known[dev][cl].load(std::memory_order_relaxed);
    if (n > 0) return n;
  }
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)cl;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)cl);
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = (size_t)smem;
  c.attrs = &at;
  c.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &c) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  if (n > 0 && dev >= 0 && dev < 64) known[dev][cl].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace
}  // namespace mix
}  // namespace gdr
