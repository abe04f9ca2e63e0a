// What the matrix products share: the 16-bit types, the activations, and the sums that
// meet in a cluster's shared memory.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe.h"
#include "moe_internal.cuh"

namespace moe {

template <bool kBf16>
__device__ __forceinline__ float to_f(uint16_t u) {
  if (kBf16) return __bfloat162float(__ushort_as_bfloat16(u));
  return __half2float(__ushort_as_half(u));
}
template <bool kBf16>
__device__ __forceinline__ uint16_t from_f(float v) {
  if (kBf16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  return __half_as_ushort(__float2half_rn(v));
}

// v sigmoid(v) and the like through one exponential (the quotient is 0 where it
// has run over); erfc keeps gelu's negative tail from cancelling.
__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case MOE_ACT_SILU: return __fdividef(v, 1.f + __expf(-v));
    case MOE_ACT_GELU: return 0.5f * v * erfcf(-v * 0.70710678118654752f);
    case MOE_ACT_GELU_TANH:
      return __fdividef(v, 1.f + __expf(-1.5957691216057308f * (v + 0.044715f * v * v * v)));
    case MOE_ACT_RELU: return v <= 0.f ? 0.f : v;  // NaN stays NaN (fmaxf returns the other operand)
    default: return v;
  }
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// (orders no memory: says that this CTA runs)
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The place in another CTA's shared memory, and a store there.
__device__ __forceinline__ uint32_t of_rank(uint32_t local, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
  return a;
}
__device__ __forceinline__ void st_cluster(uint32_t at, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t local, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

}  // namespace moe
