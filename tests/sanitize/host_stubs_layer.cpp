// Host-only stand-ins for the launchers of the steps around a layer's products
// (see host_stubs.cpp).
#include "layer_kernels.h"

namespace mxq {

hipError_t launch_rmsnorm(const NormArgs&, mxq_format, hipStream_t) { return hipErrorNoDevice; }
int64_t norm_bwd_groups(int64_t rows, int64_t) { return rows < 256 ? rows : 256; }
hipError_t launch_rmsnorm_backward(const NormBwdArgs&, hipStream_t) { return hipErrorNoDevice; }
void plan_moe(MoeArgs& a, bool) {
  a.group_tokens = 32;
  a.groups = a.T > 64 ? (a.T + 31) / 32 : 0;
}
hipError_t launch_moe_route(const MoeArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_moe_sort(const MoeArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_moe_route_backward(const RouteBwdArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_moe_dispatch(const MoeRowsArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_moe_combine(const MoeRowsArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_moe_combine_backward(const MoeRowsArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_rope_append(const RopeArgs&, hipStream_t) { return hipErrorNoDevice; }

}  // namespace mxq
