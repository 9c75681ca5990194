// Addressing of the paged NVFP4 cache shared by the kernels that write and
// read it.
#pragma once

#include "decode_kernels.h"
#include "mxq_device.h"
#include "requests.h"

namespace mxq {

// The page of cache position pos of request b, or -1: a position outside the
// table's row, or an entry outside [0, pages).
__device__ __forceinline__ int64_t page_of(const CacheArgs& c, int64_t b, int64_t pos) {
  const int64_t i = pos >> c.P_log2;
  if (pos < 0 || i >= c.width) return -1;
  const int64_t p = c.table[b * c.ld_table + i];
  return p < c.pages ? p : -1;                 // negative entries pass through
}

}  // namespace mxq
