// Checks and settings shared by the translation units of libhs.so beyond the pool itself (not part of the C ABI).
#ifndef HS_INTERNAL_HPP_
#define HS_INTERNAL_HPP_

#include <cuda_runtime.h>

#include "hs_pool.hpp"

bool hs_paged_ok(const hs_paged_rows* p);  // whether a block table's sizes and alignments are usable
bool hs_on_device(const hs_pool* p);       // whether the pool's device is the current one
int hs_launched(cudaError_t e);            // HS_OK, or HS_ERR_CUDA with the runtime's last error taken back
// The settings of hs_debug_attention: polling rounds of the attention kernels' waits, and the stall hook.
void hs_attention_waits(uint32_t* limit, int32_t* stall);

#endif  // HS_INTERNAL_HPP_
