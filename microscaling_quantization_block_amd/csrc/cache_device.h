// Addressing of the paged NVFP4 cache shared by the kernels that write and
// read it.
#pragma once

#include "decode_kernels.h"
#include "mxq_device.h"

namespace mxq {

// The request that owns query row t: the largest b with q_offsets[b] <= t,
// -1 if t lies in no request (rows before the first or behind the last).
__device__ __forceinline__ int64_t request_of(const CacheArgs& c, int64_t t) {
  if (!c.q_offsets) return t < c.B ? t : -1;
  if (t < c.q_offsets[0] || t >= c.q_offsets[c.B]) return -1;
  int64_t lo = 0, hi = c.B;                    // q_offsets[lo] <= t < q_offsets[hi]
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (c.q_offsets[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The page of cache position pos of request b, or -1: a position outside the
// table's row, or an entry outside [0, pages).
__device__ __forceinline__ int64_t page_of(const CacheArgs& c, int64_t b, int64_t pos) {
  const int64_t i = pos >> c.P_log2;
  if (pos < 0 || i >= c.width) return -1;
  const int64_t p = c.table[b * c.ld_table + i];
  return p < c.pages ? p : -1;                 // negative entries pass through
}

}  // namespace mxq
