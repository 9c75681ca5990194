// Host-side launchers of the steps around a layer's products: the norm, the
// router and the experts' rows, the rotated cache append (internal to the
// library).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "decode_kernels.h"

namespace mxq {

struct NormArgs {
  const uint16_t *x, *r, *w;    // r: nullptr without a residual
  int64_t ld_x, ld_r;
  int64_t rows, cols;
  double eps;
  uint16_t* h;                  // x + r, or nullptr
  int64_t ld_h;
  uint16_t* y;                  // or nullptr
  int64_t ld_y;
  float* rstd;                  // [rows], or nullptr
  uint8_t* codes;               // quantized output (fmt != MXQ_FMT_BF16)
  int64_t ld_codes;             // bytes
  uint8_t* scales;
  int mfma;
  float* gs;                    // NVFP4: [rows]
  uint16_t* dq;                 // the codes' values, or nullptr
  int64_t ld_dq;
};
hipError_t launch_rmsnorm(const NormArgs& a, mxq_format fmt, hipStream_t st);

struct NormBwdArgs {
  const uint16_t *dy, *h, *w, *dres;   // dres: nullptr without a residual
  int64_t ld_dy, ld_h, ld_dres;
  const float* rstd;
  int64_t rows, cols;
  uint16_t* dx;
  int64_t ld_dx;
  float* dw;                    // [cols], or nullptr
  float* part;                  // [norm_bwd_groups(rows, cols), cols] partial sums of dw
};
// Workgroups of the backward kernel, each with one partial sum of dw.
int64_t norm_bwd_groups(int64_t rows, int64_t cols);
hipError_t launch_rmsnorm_backward(const NormBwdArgs& a, hipStream_t st);

// Rows of the experts: ids [T, k] to rows ordered by (expert, token).
struct MoeArgs {
  const void* logits;           // [T, E], binary32 or BF16 (mx_moe_route)
  int f32, renorm;
  int64_t ld;
  int64_t T;
  int E, k;
  int32_t* experts;             // [T, k]: written by the router, else given
  float* weights;               // [T, k]
  int32_t *offsets;             // [E + 1]
  int32_t *row_token, *row_of;  // [T k], [T, k]
  uint16_t* counts;             // [groups, moe_pad(E)] tokens' slots of each expert
  int64_t groups, group_tokens;
};
constexpr int MOE_EXPERTS = 1024, MOE_TOPK = 64;
// Experts of a row of counts: whole 16-byte loads.
inline int64_t moe_pad(int E) { return (E + 7) / 8 * 8; }
// Sets a.groups (0: one workgroup does it all, without counts) and a.group_tokens.
void plan_moe(MoeArgs& a, bool routed);
hipError_t launch_moe_route(const MoeArgs& a, hipStream_t st);
hipError_t launch_moe_sort(const MoeArgs& a, hipStream_t st);

struct RouteBwdArgs {
  const float* dweights;        // [T, k]
  const void* logits;
  int f32, renorm;
  int64_t ld, T;
  int E, k;
  const int32_t* experts;
  const float* weights;
  void* dlogits;                // as logits
  int64_t ld_d;
};
hipError_t launch_moe_route_backward(const RouteBwdArgs& a, hipStream_t st);

struct MoeRowsArgs {
  int64_t T, cols, M;           // tokens, values of a row, rows of the experts
  int k;
  const int32_t* row_of;        // [T, k]
  const float* weights;         // [T, k], or nullptr: ones
  const uint16_t* x;            // tokens' rows in
  uint16_t* out;                // tokens' rows out
  int64_t ld_x, ld_out;
  const uint16_t* rows;         // experts' rows in
  uint16_t* to_rows;            // experts' rows out
  int64_t ld_rows, ld_to;
  float* dweights;              // [T, k]
};
hipError_t launch_moe_dispatch(const MoeRowsArgs& a, hipStream_t st);
hipError_t launch_moe_combine(const MoeRowsArgs& a, hipStream_t st);
hipError_t launch_moe_combine_backward(const MoeRowsArgs& a, hipStream_t st);

struct RopeArgs {
  AppendArgs p;                 // k, v and the cache
  const uint16_t* q;
  int Hq;
  int64_t q_token, q_head;      // strides, elements
  uint16_t* q_out;
  int64_t o_token, o_head;
  const float* inv_freq;        // [rot / 2]
  int rot, interleaved;
  double factor;
  int split;                    // waves of a token (set by the launcher)
};
hipError_t launch_rope_append(const RopeArgs& a, hipStream_t st);

}  // namespace mxq
