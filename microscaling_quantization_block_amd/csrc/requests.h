// Which rows of a call belong to which request: the one rule that every kernel
// of the cache goes by (plain code, the host tests run it too).
#pragma once

#include "decode_kernels.h"

namespace mxq {

// The rows of request b among the call's T: the first one and their number, 0
// where the offsets do not lie in [0, T] in order.
struct RequestRows {
  int begin, len;
};
__host__ __device__ inline RequestRows request_rows(const CacheArgs& c, int64_t b, int64_t T) {
  RequestRows r = {(int)b, 1};
  if (c.q_offsets) {
    const int begin = c.q_offsets[b], end = c.q_offsets[b + 1];
    r.begin = begin;
    r.len = begin >= 0 && end <= T && end > begin ? end - begin : 0;
  }
  return r;
}

// The request that owns row t and its rows: the largest b with q_offsets[b] <= t,
// -1 if t lies in no request (rows before the first or behind the last, and those
// whose request has no rows by the rule above).
__host__ __device__ inline int64_t request_of(const CacheArgs& c, int64_t t, int64_t T, RequestRows& rows) {
  rows = {(int)t, 1};
  if (!c.q_offsets) return t < c.B ? t : -1;
  if (t < c.q_offsets[0] || t >= c.q_offsets[c.B]) return -1;
  int64_t lo = 0, hi = c.B;                    // q_offsets[lo] <= t < q_offsets[hi]
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (c.q_offsets[mid] <= t) lo = mid;
    else hi = mid;
  }
  rows = request_rows(c, lo, T);
  return rows.len ? lo : -1;
}

}  // namespace mxq
