// Host-only stand-ins for the launchers of the decode step (see host_stubs.cpp).
#include "decode_kernels.h"

namespace mxq {

hipError_t launch_nvfp4_gemv(const GemvArgs&, GemvScales, bool, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_cache_append(const AppendArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_attention(const AttnArgs&, const AttnPlan&, hipStream_t) { return hipErrorNoDevice; }

}  // namespace mxq
