// sv_cluster.cuh - thread-block cluster helpers (sm_103a): rank queries, the
// cluster barrier and stores into the shared memory of another CTA of the
// cluster.  Device code only.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "sv_ptx.cuh"

namespace sv {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}
// Barrier over every thread of the cluster.  What any of them wrote before it
// (shared, distributed shared or global memory) is visible to all after it;
// read such global data with __ldcg.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of `p` (a shared variable of this CTA) in the CTA of rank r.
__device__ __forceinline__ uint32_t cluster_map(const void* p, uint32_t r) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(r));
  return a;
}
__device__ __forceinline__ void cluster_st(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_st64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

}  // namespace sv
