// C ABI of the steps around a layer's products (include/mxq_layer.h): argument
// validation on the host, then kernel launches on the caller's stream, as in api.cpp.

#include <math.h>

#include "api_cache.h"
#include "layer_kernels.h"
#include "mxq_layer.h"

using mxq::aligned;
using mxq::aligned16;
using mxq::fail;
using mxq::hip_status;
using mxq::I31;
using mxq::ok;

namespace {

hipStream_t S(void* s) { return reinterpret_cast<hipStream_t>(s); }

constexpr int64_t NORM_COLS = 32768;

// [rows, cols] BF16 with a row stride in elements
mxq_status check_matrix(const char* fn, const char* name, const uint16_t* p, int64_t ld, int64_t cols) {
  if (!p) return fail(MXQ_EINVAL, "%s: %s is NULL", fn, name);
  if (ld < cols) return fail(MXQ_EINVAL, "%s: leading dimension of %s smaller than the row", fn, name);
  if (!aligned16(p) || ld % 8) return fail(MXQ_EALIGN, "%s: %s 16-byte aligned, its stride a multiple of 8", fn, name);
  return MXQ_OK;
}

mxq_status check_norm_shape(const char* fn, int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return fail(MXQ_EINVAL, "%s: negative size", fn);
  if (cols % 8) return fail(MXQ_ESHAPE, "%s: cols %% 8 == 0 (cols=%lld)", fn, (long long)cols);
  if (cols > NORM_COLS) return fail(MXQ_EUNSUPPORTED, "%s: cols up to %lld", fn, (long long)NORM_COLS);
  if (rows >= I31) return fail(MXQ_EUNSUPPORTED, "%s: too many rows for one call", fn);
  return MXQ_OK;
}

}  // namespace

extern "C" {

mxq_status mx_rmsnorm(const uint16_t* x, int64_t ld_x, const uint16_t* residual, int64_t ld_r,
                      const uint16_t* weight, int64_t rows, int64_t cols, float eps, uint16_t* h, int64_t ld_h,
                      uint16_t* y, int64_t ld_y, float* rstd, mxq_format fmt, mxq_scale_layout layout,
                      uint8_t* codes, int64_t ld_codes, void* scales, float* gscales, uint16_t* dq, int64_t ld_dq,
                      void* stream) {
  const char* fn = "mx_rmsnorm";
  mxq_status s = check_norm_shape(fn, rows, cols);
  if (s != MXQ_OK) return s;
  if (!(eps >= 0.0f) || !isfinite(eps)) return fail(MXQ_EINVAL, "%s: eps must be finite and not negative", fn);
  // the enumerators as numbers: a value the enum does not have must reach the checks
  const int f = static_cast<int>(fmt), lay = static_cast<int>(layout);
  const int64_t block = f == MXQ_FMT_MXFP8 ? 32 : f == MXQ_FMT_NVFP4 ? 16 : f == MXQ_FMT_BF16 ? 8 : 128;
  if (f < MXQ_FMT_MXFP8 || f > MXQ_FMT_FP8_B128_F32) return fail(MXQ_EINVAL, "%s: bad format", fn);
  if (lay != MXQ_LAYOUT_LINEAR && lay != MXQ_LAYOUT_MFMA) return fail(MXQ_EINVAL, "%s: bad scale layout", fn);
  const bool quantize = f != MXQ_FMT_BF16, mfma = lay == MXQ_LAYOUT_MFMA;
  if (mfma && f != MXQ_FMT_MXFP8 && f != MXQ_FMT_NVFP4)
    return fail(MXQ_EUNSUPPORTED, "%s: MFMA scales are for MXFP8 and NVFP4", fn);
  if (cols % block) return fail(MXQ_ESHAPE, "%s: cols must be a multiple of the format's block (%lld)", fn, (long long)block);
  if (mfma && (rows % 32 || cols % (4 * block)))
    return fail(MXQ_ESHAPE, "%s: MFMA scales need rows %% 32 == 0 and cols %% %lld == 0", fn, (long long)(4 * block));
  if (rows == 0 || cols == 0) return ok();

  if ((s = check_matrix(fn, "x", x, ld_x, cols)) != MXQ_OK) return s;
  if ((s = check_matrix(fn, "weight", weight, cols, cols)) != MXQ_OK) return s;
  if (residual && (s = check_matrix(fn, "residual", residual, ld_r, cols)) != MXQ_OK) return s;
  if (h && !residual) return fail(MXQ_EINVAL, "%s: h without a residual is x", fn);
  if (h && (s = check_matrix(fn, "h", h, ld_h, cols)) != MXQ_OK) return s;
  if (!y && !quantize) return fail(MXQ_EINVAL, "%s: y is NULL", fn);
  if (y && (s = check_matrix(fn, "y", y, ld_y, cols)) != MXQ_OK) return s;
  if (!aligned(rstd, 4)) return fail(MXQ_EALIGN, "%s: rstd 4-byte aligned", fn);
  if (!quantize) {
    if (codes || scales || gscales || dq) return fail(MXQ_EINVAL, "%s: BF16 output has no codes", fn);
  } else {
    if (!codes || !scales || (f == MXQ_FMT_NVFP4 && !gscales)) return fail(MXQ_EINVAL, "%s: null pointer", fn);
    if (f != MXQ_FMT_NVFP4 && gscales) return fail(MXQ_EINVAL, "%s: gscales are NVFP4's", fn);
    if (ld_codes < (f == MXQ_FMT_NVFP4 ? cols / 2 : cols))
      return fail(MXQ_EINVAL, "%s: leading dimension of the codes smaller than the row", fn);
    if (!aligned16(codes) || ld_codes % 16 || !aligned(gscales, 4) || (f == MXQ_FMT_FP8_B128_F32 && !aligned(scales, 4)))
      return fail(MXQ_EALIGN, "%s: codes 16-byte aligned, ld_codes %% 16 == 0, float scales 4-byte aligned", fn);
    if (dq && (s = check_matrix(fn, "dq", dq, ld_dq, cols)) != MXQ_OK) return s;
  }

  mxq::NormArgs a = {};
  a.x = x;
  a.r = residual;
  a.w = weight;
  a.ld_x = ld_x;
  a.ld_r = ld_r;
  a.rows = rows;
  a.cols = cols;
  a.eps = eps;
  a.h = h;
  a.ld_h = ld_h;
  a.y = y;
  a.ld_y = ld_y;
  a.rstd = rstd;
  a.codes = codes;
  a.ld_codes = ld_codes;
  a.scales = static_cast<uint8_t*>(scales);
  a.mfma = mfma;
  a.gs = gscales;
  a.dq = dq;
  a.ld_dq = ld_dq;
  return hip_status(mxq::launch_rmsnorm(a, static_cast<mxq_format>(f), S(stream)), fn);
}

int64_t mx_rmsnorm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || cols > NORM_COLS || rows >= I31) return 0;      // nothing to do, or refused
  return mxq::norm_bwd_groups(rows, cols) * cols * 4;
}

mxq_status mx_rmsnorm_backward(const uint16_t* dy, int64_t ld_dy, const uint16_t* h, int64_t ld_h,
                               const uint16_t* weight, const float* rstd, const uint16_t* dresidual,
                               int64_t ld_dr, int64_t rows, int64_t cols, uint16_t* dx, int64_t ld_dx,
                               float* dweight, void* workspace, int64_t workspace_bytes, void* stream) {
  const char* fn = "mx_rmsnorm_backward";
  mxq_status s = check_norm_shape(fn, rows, cols);
  if (s != MXQ_OK) return s;
  if (cols == 0) return ok();
  if (!aligned16(dweight)) return fail(MXQ_EALIGN, "%s: dweight 16-byte aligned", fn);
  if (rows == 0 && !dweight) return ok();
  if (rows > 0) {
    if ((s = check_matrix(fn, "dy", dy, ld_dy, cols)) != MXQ_OK) return s;
    if ((s = check_matrix(fn, "h", h, ld_h, cols)) != MXQ_OK) return s;
    if ((s = check_matrix(fn, "weight", weight, cols, cols)) != MXQ_OK) return s;
    if ((s = check_matrix(fn, "dx", dx, ld_dx, cols)) != MXQ_OK) return s;
    if (dresidual && (s = check_matrix(fn, "dresidual", dresidual, ld_dr, cols)) != MXQ_OK) return s;
    if (!rstd) return fail(MXQ_EINVAL, "%s: rstd is NULL", fn);
    if (!aligned(rstd, 4)) return fail(MXQ_EALIGN, "%s: rstd 4-byte aligned", fn);
  }
  if (dweight && rows > 0) {
    const int64_t need = mx_rmsnorm_backward_workspace(rows, cols);
    if (!workspace || workspace_bytes < need)
      return fail(MXQ_EINVAL, "%s: the workspace needs %lld bytes", fn, (long long)need);
    if (!aligned16(workspace)) return fail(MXQ_EALIGN, "%s: workspace 16-byte aligned", fn);
  }
  mxq::NormBwdArgs a = {};
  a.dy = dy;
  a.h = h;
  a.w = weight;
  a.dres = dresidual;
  a.ld_dy = ld_dy;
  a.ld_h = ld_h;
  a.ld_dres = ld_dr;
  a.rstd = rstd;
  a.rows = rows;
  a.cols = cols;
  a.dx = dx;
  a.ld_dx = ld_dx;
  a.dw = dweight;
  a.part = static_cast<float*>(workspace);
  return hip_status(mxq::launch_rmsnorm_backward(a, S(stream)), fn);
}

}  // extern "C"
