// Loads of the caller's index arrays (selections, positions, lengths, resident maps, slot lists).
#pragma once

#include <cstdint>

namespace hs {

// `.cv` fetches afresh, so a stale L2 copy of a host-memory line is never used and these arrays may live in device memory
// or in mapped page-locked host memory, read over the host link without a separate copy. Volatile: it stays behind the
// griddepcontrol.wait that the kernel starts with (a volatile asm too), until which the kernel that writes the array may
// still run; without it the compiler may load ahead of that wait.
__device__ __forceinline__ int32_t ld_fresh(const int32_t* p) {
  int32_t v;
  asm volatile("ld.global.cv.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

}  // namespace hs
