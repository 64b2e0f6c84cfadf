// Thread-block clusters of the operators around the GEMMs: their size, and the cluster
// barrier in halves.  Beside common.cuh, whose text the GEMMs' committed DRAM captures
// are bound to.
#pragma once

#include <cstdint>

namespace mg {

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
// All threads of the cluster arrive, then all wait.  Relaxed: to know that the blocks
// run, without ordering what they wrote.
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

}  // namespace mg
