// Where the entries of a selection find their rows (not part of the C ABI).
#ifndef HS_SOURCE_HPP_
#define HS_SOURCE_HPP_

#include <cstddef>
#include <cstdint>

#include "hs_pool.hpp"

// Where the entries of a selection find their rows: entry e >= 0 is row e of its request in `rows` (a hot slot, or a token
// of the history), an entry <= -2 row -2 - e of `resident`, if there is one; anything else is no row.
struct RowSource {
  const uint8_t* rows;      // request 0's
  int64_t req_stride;       // bytes between requests
  int32_t limit;            // rows 0 .. limit - 1 of a request
  const uint8_t* resident;  // or nullptr
  int64_t resident_count;
};
#ifdef __CUDACC__
__device__ __forceinline__ const uint8_t* row_at(const RowSource& s, uint32_t request, int32_t e, int row_bytes) {
  if (e >= 0) return e < s.limit ? s.rows + (size_t)request * (size_t)s.req_stride + (size_t)e * row_bytes : nullptr;
  const int64_t r = -2ll - e;
  return e <= -2 && s.resident && r < s.resident_count ? s.resident + (size_t)r * row_bytes : nullptr;
}
#endif
RowSource hs_slot_rows(const hs_pool* p, int32_t layer, const void* resident_rows, int64_t resident_count);
RowSource hs_history_rows(const hs_pool* p, int32_t layer);

#endif  // HS_SOURCE_HPP_
