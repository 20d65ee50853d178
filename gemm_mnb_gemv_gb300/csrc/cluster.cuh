// Thread-block clusters: the barrier and loads from another CTA's shared memory.
#pragma once

#include <stdint.h>

namespace mnb {

__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// All threads of all CTAs of the cluster call both, in this order.  What a thread wrote to shared memory before arriving
// is visible to every thread behind its wait; a CTA whose memory others read must not end before they have arrived.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Address of this CTA's shared-memory address `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 cluster_ld_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void cluster_st_u64(uint32_t addr, uint32_t lo, uint32_t hi) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(lo), "r"(hi) : "memory");
}
__device__ __forceinline__ void cluster_st_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// Sum over the CTAs, in their order, of the float4 at this CTA's address; eight loads in flight.
__device__ __forceinline__ float4 cluster_sum_f4(uint32_t addr, int cluster) {
  float4 v = make_float4(0, 0, 0, 0);
  for (int c0 = 0; c0 < cluster; c0 += 8) {
    float4 o[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      o[c] = make_float4(0, 0, 0, 0);
      if (c0 + c < cluster) o[c] = cluster_ld_f4(cluster_map(addr, c0 + c));
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) v.x += o[c].x, v.y += o[c].y, v.z += o[c].z, v.w += o[c].w;
  }
  return v;
}
}  // namespace mnb
