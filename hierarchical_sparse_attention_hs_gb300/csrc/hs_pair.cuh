// Helpers of the kernels in which a pair of CTAs runs its tensor-core work together (cta_group::2, sm_103a).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
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

// A box at column block `blk` and row `row` into this CTA's shared memory; its bytes count on a barrier of the pair's
// first CTA.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int blk, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
      "%5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(row), "r"(blk)
      : "memory");
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeFn encoder() {
  static std::atomic<EncodeFn> fn{nullptr};
  EncodeFn f = fn.load(std::memory_order_acquire);
  if (f) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  f = reinterpret_cast<EncodeFn>(p);
  fn.store(f, std::memory_order_release);
  return f;
}
// Rows of 576 bf16 values as (column, row, 64-column block): boxes of 64 columns x `box` rows x `blocks` blocks, which lie
// block by block in shared memory, 128-byte swizzle, zeros outside.
inline bool make_map(EncodeFn f, CUtensorMap* m, const void* rows, uint64_t count, uint32_t box, uint32_t blocks) {
  const cuuint64_t dims[3] = {64, count, 9}, strides[2] = {1152, 128};
  const cuuint32_t boxes[3] = {64, box, blocks}, steps[3] = {1, 1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(rows), dims, strides, boxes, steps,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace hs
