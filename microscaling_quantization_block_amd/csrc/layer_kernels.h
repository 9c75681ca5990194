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

}  // namespace mxq
