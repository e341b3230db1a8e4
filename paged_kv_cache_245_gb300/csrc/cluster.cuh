// cluster.cuh -- thread-block clusters: the barrier, and reads of another CTA's
// shared memory.
#pragma once

#include <stdint.h>

#include "pkv_device.cuh"

namespace pkv {

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// The shared-memory address `of` in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t in_cta(const void* of, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(of)), "r"(rank));
  return a;
}

__device__ __forceinline__ int32_t ld_cluster_s32(uint32_t a) {
  int32_t x;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(a) : "memory");
  return x;
}

__device__ __forceinline__ float2 ld_cluster_f2(uint32_t a) {
  float2 x;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(a) : "memory");
  return x;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t a) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(a)
               : "memory");
  return x;
}

}  // namespace pkv
