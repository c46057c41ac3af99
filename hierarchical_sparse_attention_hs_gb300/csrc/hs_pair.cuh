// Helpers of the kernels in which a pair of CTAs runs its tensor-core work together (cta_group::2, sm_103a).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "hs_tcgen05.cuh"

namespace hs {

// Shared-memory matrix descriptor, 128-byte swizzle. K-major: 8-row groups 1024 bytes apart (lbo unused). MN-major: `lbo`
// between 64-element runs along M or N, 1024 bytes between 8-deep groups along K.
__device__ __forceinline__ uint64_t sdesc128(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ void mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// arrive on the barrier at this offset in both CTAs (`mask`: their bits of the cluster) once every MMA issued so far has finished
__device__ __forceinline__ void commit2(uint64_t* b, uint32_t mask = 3) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(su32(b)),
      "h"((uint16_t)mask)
      : "memory");
}
// Arrive on a barrier of the pair's first CTA. What it orders are this thread's tensor-memory reads and shared-memory
// writes before the MMAs that the issuer starts after its wait, which the tcgen05 and proxy fences before it cover; a
// release of cluster scope on top would cost about 870 cycles an arrival (measured).
__device__ __forceinline__ void arrive_lead(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void arrive_lead(uint32_t addr, uint32_t count) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0], %1;" ::"r"(addr), "r"(count) : "memory");
}
// One lane of a converged warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
  return p != 0;
}

}  // namespace hs
