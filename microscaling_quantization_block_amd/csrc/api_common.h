// What the sources of the C ABI share: the thread-local error text (defined in
// api.cpp) and small argument helpers.  Internal to the library.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq.h"

namespace mxq {

// Records the message for mxq_last_error() and returns s.
mxq_status fail(mxq_status s, const char* fmt, ...);
// Clears the message and returns MXQ_OK.
mxq_status ok();
mxq_status hip_status(hipError_t e, const char* what);

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace mxq
