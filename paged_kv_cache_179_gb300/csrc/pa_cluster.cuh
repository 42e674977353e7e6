// pa_cluster.cuh -- thread-block clusters: ranks, the barrier and addresses in
// distributed shared memory.
#pragma once

#include "pa_ptx.cuh"

namespace pa {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// The cluster's barrier, in two halves, by all its threads; shared memory written
// before the arrival is seen after the wait.  The .aligned forms want a warp's
// threads there together, which a loop or a branch before them does not give.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// What p (in this CTA's shared memory) is in CTA `rank`'s.
__device__ __forceinline__ uint32_t in_cluster(const void* p, uint32_t rank) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  return at;
}

}  // namespace pa
