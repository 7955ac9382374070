// tcgen05.cuh -- pieces of the fifth-generation tensor-core path that the
// products share: the shared-memory matrix descriptor, commits and fences.
#pragma once

#include "common.cuh"

namespace qamw {

// Shared-memory matrix descriptor of a K-major tile with the 128-byte swizzle:
// start address >> 4 (bits 0-13), leading-dimension offset 16 B (bits 16-29,
// unused for this layout), stride between 8-row groups 1024 B (bits 32-45),
// descriptor version 1 (bits 46-47), base offset 0, layout type 2 = 128-byte
// swizzle (bits 61-63).
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Arrive on the mbarrier once every MMA this thread issued so far has completed.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

}  // namespace qamw
