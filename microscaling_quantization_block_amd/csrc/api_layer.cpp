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

// Sizes of the experts' rows.
mxq_status check_slots(const char* fn, int64_t tokens, int topk) {
  if (tokens < 0) return fail(MXQ_EINVAL, "%s: negative size", fn);
  if (topk < 1 || topk > mxq::MOE_TOPK) return fail(MXQ_EINVAL, "%s: topk must be 1 to %d (topk=%d)", fn, mxq::MOE_TOPK, topk);
  // 32-bit grids: up to a workgroup of 256 lanes per token, one per four slots (rounded up)
  if (tokens >= (1 << 24) || tokens * topk > (1 << 26) - 4)
    return fail(MXQ_EUNSUPPORTED, "%s: too many tokens for one call (below 2^24, at most 2^26 - 4 slots)", fn);
  return MXQ_OK;
}

mxq_status check_experts(const char* fn, int64_t tokens, int num_experts, int topk) {
  const mxq_status s = check_slots(fn, tokens, topk);
  if (s != MXQ_OK) return s;
  if (num_experts < 1) return fail(MXQ_EINVAL, "%s: no experts", fn);
  if (num_experts > mxq::MOE_EXPERTS)
    return fail(MXQ_EUNSUPPORTED, "%s: up to %d experts (num_experts=%d)", fn, mxq::MOE_EXPERTS, num_experts);
  if (topk > num_experts) return fail(MXQ_ESHAPE, "%s: topk exceeds the experts (%d, %d)", fn, topk, num_experts);
  return MXQ_OK;
}

mxq_status check_logits(const char* fn, const char* name, const void* p, bool f32, int64_t ld, int num_experts) {
  if (!p) return fail(MXQ_EINVAL, "%s: %s is NULL", fn, name);
  if (ld < num_experts) return fail(MXQ_EINVAL, "%s: leading dimension of %s smaller than the row", fn, name);
  if (ld >= I31) return fail(MXQ_EUNSUPPORTED, "%s: leading dimension of %s too large", fn, name);
  if (!aligned(p, f32 ? 4 : 2)) return fail(MXQ_EALIGN, "%s: %s is not aligned to its type", fn, name);
  return MXQ_OK;
}

// The outputs of the sort, its workspace and its plan.
mxq_status check_sort(const char* fn, mxq::MoeArgs& a, bool routed, void* workspace, int64_t workspace_bytes) {
  if (!a.offsets) return fail(MXQ_EINVAL, "%s: offsets is NULL", fn);
  if (a.T > 0 && (!a.experts || !a.row_token || !a.row_of)) return fail(MXQ_EINVAL, "%s: null pointer", fn);
  if (!aligned(a.offsets, 4) || !aligned(a.experts, 4) || !aligned(a.row_token, 4) || !aligned(a.row_of, 4) ||
      !aligned(a.weights, 4))
    return fail(MXQ_EALIGN, "%s: arrays 4-byte aligned", fn);
  mxq::plan_moe(a, routed);
  const int64_t need = a.groups * mxq::moe_pad(a.E) * 2;
  if (need) {
    if (!workspace || workspace_bytes < need)
      return fail(MXQ_EINVAL, "%s: the workspace needs %lld bytes", fn, (long long)need);
    if (!aligned16(workspace)) return fail(MXQ_EALIGN, "%s: workspace 16-byte aligned", fn);
    a.counts = static_cast<uint16_t*>(workspace);
  }
  return MXQ_OK;
}

// Sizes, row_of and the matrices of a call on the experts' rows.  Sets nothing to do where there is nothing.
mxq_status check_rows_call(const char* fn, const mxq::MoeRowsArgs& a) {
  const mxq_status s = check_slots(fn, a.T, a.k);
  if (s != MXQ_OK) return s;
  if (a.cols < 0 || a.M < 0) return fail(MXQ_EINVAL, "%s: negative size", fn);
  if (a.cols % 8) return fail(MXQ_ESHAPE, "%s: cols %% 8 == 0 (cols=%lld)", fn, (long long)a.cols);
  if (a.cols >= (1 << 26)) return fail(MXQ_EUNSUPPORTED, "%s: cols below 2^26", fn);
  if (a.M >= I31) return fail(MXQ_EUNSUPPORTED, "%s: too many rows", fn);
  if (a.T == 0) return MXQ_OK;
  if (!a.row_of) return fail(MXQ_EINVAL, "%s: row_of is NULL", fn);
  if (!aligned(a.row_of, 4) || !aligned(a.weights, 4) || !aligned(a.dweights, 4))
    return fail(MXQ_EALIGN, "%s: arrays 4-byte aligned", fn);
  return MXQ_OK;
}

}  // namespace

extern "C" {

mxq_status mx_rmsnorm(const uint16_t* x, int64_t ld_x, const uint16_t* residual, int64_t ld_r,
                      const uint16_t* weight, int64_t rows, int64_t cols, double eps, uint16_t* h, int64_t ld_h,
                      uint16_t* y, int64_t ld_y, float* rstd, mxq_format fmt, mxq_scale_layout layout,
                      uint8_t* codes, int64_t ld_codes, void* scales, float* gscales, uint16_t* dq, int64_t ld_dq,
                      void* stream) {
  const char* fn = "mx_rmsnorm";
  mxq_status s = check_norm_shape(fn, rows, cols);
  if (s != MXQ_OK) return s;
  if (!(eps >= 0.0) || !isfinite(eps)) return fail(MXQ_EINVAL, "%s: eps must be finite and not negative", fn);
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
    // a block of NVFP4 is 8 bytes (the quantizer's rule), of MXFP8 32; the kernel stores whole words
    const int64_t unit = f == MXQ_FMT_NVFP4 ? 8 : 16;
    if (!aligned16(codes) || ld_codes % unit || !aligned(gscales, 4) || (f == MXQ_FMT_FP8_B128_F32 && !aligned(scales, 4)))
      return fail(MXQ_EALIGN, "%s: codes 16-byte aligned, ld_codes %% %d == 0, float scales 4-byte aligned", fn, (int)unit);
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

int64_t mx_moe_workspace(int64_t tokens, int32_t num_experts, int32_t topk) {
  if (tokens <= 0 || tokens >= (1 << 24) || topk < 1 || topk > mxq::MOE_TOPK || num_experts < 1 ||
      num_experts > mxq::MOE_EXPERTS)
    return 0;                                  // nothing to do, or refused
  mxq::MoeArgs a = {};
  a.T = tokens;
  a.E = num_experts;
  a.k = topk;
  int64_t groups = 0;
  for (const bool routed : {false, true}) {
    mxq::plan_moe(a, routed);
    if (a.groups > groups) groups = a.groups;
  }
  return groups * mxq::moe_pad(num_experts) * 2;
}

mxq_status mx_moe_route(const void* logits, int32_t logits_f32, int64_t ld, int64_t tokens, int32_t num_experts,
                        int32_t topk, int32_t renormalize, int32_t* experts, float* weights, int32_t* offsets,
                        int32_t* row_token, int32_t* row_of, void* workspace, int64_t workspace_bytes, void* stream) {
  const char* fn = "mx_moe_route";
  mxq_status s = check_experts(fn, tokens, num_experts, topk);
  if (s != MXQ_OK) return s;
  if (tokens > 0) {
    if ((s = check_logits(fn, "logits", logits, logits_f32, ld, num_experts)) != MXQ_OK) return s;
    if (!weights) return fail(MXQ_EINVAL, "%s: weights is NULL", fn);
  }
  mxq::MoeArgs a = {};
  a.logits = logits;
  a.f32 = logits_f32 != 0;
  a.renorm = renormalize != 0;
  a.ld = ld;
  a.T = tokens;
  a.E = num_experts;
  a.k = topk;
  a.experts = experts;
  a.weights = weights;
  a.offsets = offsets;
  a.row_token = row_token;
  a.row_of = row_of;
  if ((s = check_sort(fn, a, true, workspace, workspace_bytes)) != MXQ_OK) return s;
  return hip_status(mxq::launch_moe_route(a, S(stream)), fn);
}

mxq_status mx_moe_sort(const int32_t* experts, int64_t tokens, int32_t num_experts, int32_t topk, int32_t* offsets,
                       int32_t* row_token, int32_t* row_of, void* workspace, int64_t workspace_bytes, void* stream) {
  const char* fn = "mx_moe_sort";
  mxq_status s = check_experts(fn, tokens, num_experts, 1);
  if (s != MXQ_OK || (s = check_slots(fn, tokens, topk)) != MXQ_OK) return s;
  mxq::MoeArgs a = {};
  a.T = tokens;
  a.E = num_experts;
  a.k = topk;
  a.experts = const_cast<int32_t*>(experts);   // read only
  a.offsets = offsets;
  a.row_token = row_token;
  a.row_of = row_of;
  if ((s = check_sort(fn, a, false, workspace, workspace_bytes)) != MXQ_OK) return s;
  return hip_status(mxq::launch_moe_sort(a, S(stream)), fn);
}

mxq_status mx_moe_route_backward(const float* dweights, const void* logits, int32_t logits_f32, int64_t ld,
                                 int64_t tokens, int32_t num_experts, int32_t topk, int32_t renormalize,
                                 const int32_t* experts, const float* weights, void* dlogits, int64_t ld_d,
                                 void* stream) {
  const char* fn = "mx_moe_route_backward";
  mxq_status s = check_experts(fn, tokens, num_experts, topk);
  if (s != MXQ_OK) return s;
  if (tokens == 0) return ok();
  if ((s = check_logits(fn, "logits", logits, logits_f32, ld, num_experts)) != MXQ_OK) return s;
  if ((s = check_logits(fn, "dlogits", dlogits, logits_f32, ld_d, num_experts)) != MXQ_OK) return s;
  if (!dweights || !experts || !weights) return fail(MXQ_EINVAL, "%s: null pointer", fn);
  if (!aligned(dweights, 4) || !aligned(experts, 4) || !aligned(weights, 4))
    return fail(MXQ_EALIGN, "%s: arrays 4-byte aligned", fn);
  mxq::RouteBwdArgs a = {};
  a.dweights = dweights;
  a.logits = logits;
  a.f32 = logits_f32 != 0;
  a.renorm = renormalize != 0;
  a.ld = ld;
  a.T = tokens;
  a.E = num_experts;
  a.k = topk;
  a.experts = experts;
  a.weights = weights;
  a.dlogits = dlogits;
  a.ld_d = ld_d;
  return hip_status(mxq::launch_moe_route_backward(a, S(stream)), fn);
}

mxq_status mx_moe_dispatch(const uint16_t* x, int64_t ld_x, int64_t tokens, int64_t cols, const int32_t* row_of,
                           int32_t topk, uint16_t* rows, int64_t ld_rows, int64_t num_rows, void* stream) {
  const char* fn = "mx_moe_dispatch";
  mxq::MoeRowsArgs a = {};
  a.T = tokens;
  a.cols = cols;
  a.M = num_rows;
  a.k = topk;
  a.row_of = row_of;
  a.x = x;
  a.ld_x = ld_x;
  a.to_rows = rows;
  a.ld_to = ld_rows;
  mxq_status s = check_rows_call(fn, a);
  if (s != MXQ_OK) return s;
  if (tokens == 0 || cols == 0 || num_rows == 0) return ok();
  if ((s = check_matrix(fn, "x", x, ld_x, cols)) != MXQ_OK) return s;
  if ((s = check_matrix(fn, "rows", rows, ld_rows, cols)) != MXQ_OK) return s;
  return hip_status(mxq::launch_moe_dispatch(a, S(stream)), fn);
}

mxq_status mx_moe_combine(const uint16_t* rows, int64_t ld_rows, int64_t num_rows, const int32_t* row_of,
                          const float* weights, int64_t tokens, int64_t cols, int32_t topk, uint16_t* out,
                          int64_t ld_out, void* stream) {
  const char* fn = "mx_moe_combine";
  mxq::MoeRowsArgs a = {};
  a.T = tokens;
  a.cols = cols;
  a.M = num_rows;
  a.k = topk;
  a.row_of = row_of;
  a.weights = weights;
  a.rows = rows;
  a.ld_rows = ld_rows;
  a.out = out;
  a.ld_out = ld_out;
  mxq_status s = check_rows_call(fn, a);
  if (s != MXQ_OK) return s;
  if (tokens == 0 || cols == 0) return ok();
  if (num_rows > 0 && (s = check_matrix(fn, "rows", rows, ld_rows, cols)) != MXQ_OK) return s;
  if ((s = check_matrix(fn, "out", out, ld_out, cols)) != MXQ_OK) return s;
  return hip_status(mxq::launch_moe_combine(a, S(stream)), fn);
}

mxq_status mx_moe_combine_backward(const uint16_t* dout, int64_t ld_dout, const uint16_t* rows, int64_t ld_rows,
                                   int64_t num_rows, const int32_t* row_of, const float* weights, int64_t tokens,
                                   int64_t cols, int32_t topk, uint16_t* drows, int64_t ld_drows, float* dweights,
                                   void* stream) {
  const char* fn = "mx_moe_combine_backward";
  mxq::MoeRowsArgs a = {};
  a.T = tokens;
  a.cols = cols;
  a.M = num_rows;
  a.k = topk;
  a.row_of = row_of;
  a.weights = weights;
  a.x = dout;
  a.ld_x = ld_dout;
  a.rows = rows;
  a.ld_rows = ld_rows;
  a.to_rows = drows;
  a.ld_to = ld_drows;
  a.dweights = dweights;
  mxq_status s = check_rows_call(fn, a);
  if (s != MXQ_OK) return s;
  if (tokens == 0) return ok();
  if (!weights || !dweights) return fail(MXQ_EINVAL, "%s: null pointer", fn);
  if (cols > 0 && num_rows > 0) {
    if ((s = check_matrix(fn, "dout", dout, ld_dout, cols)) != MXQ_OK) return s;
    if ((s = check_matrix(fn, "rows", rows, ld_rows, cols)) != MXQ_OK) return s;
    if ((s = check_matrix(fn, "drows", drows, ld_drows, cols)) != MXQ_OK) return s;
  }
  return hip_status(mxq::launch_moe_combine_backward(a, S(stream)), fn);
}

mxq_status nvfp4_rope_append(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, int32_t num_q_heads,
                             const uint16_t* k, int64_t k_token_stride, int64_t k_head_stride, const uint16_t* v,
                             int64_t v_token_stride, int64_t v_head_stride, int64_t tokens, const mxq_cache* cache,
                             const int32_t* block_table, int64_t ld_table, int64_t table_width,
                             const int32_t* seq_lens, const int32_t* q_offsets, int64_t num_requests,
                             const float* inv_freq, int32_t rotary_dim, int32_t interleaved, double factor,
                             uint16_t* q_out, int64_t out_token_stride, int64_t out_head_stride, uint16_t* k_dq,
                             uint16_t* v_dq, void* stream) {
  const char* fn = "nvfp4_rope_append";
  mxq::RopeArgs a = {};
  mxq_status s = mxq::cache_args(fn, cache, block_table, ld_table, table_width, seq_lens, q_offsets, num_requests, tokens,
                                 &a.p.c);
  if (s != MXQ_OK) return s;
  const int D = cache->head_dim;
  if (num_q_heads < 1 || num_q_heads > 32767) return fail(MXQ_EINVAL, "%s: num_q_heads must be 1 to 32767", fn);
  if (rotary_dim < 16 || rotary_dim > D || rotary_dim % 16)
    return fail(MXQ_ESHAPE, "%s: rotary_dim must be a multiple of 16 up to head_dim (%d, %d)", fn, rotary_dim, D);
  if (!isfinite(factor)) return fail(MXQ_EINVAL, "%s: factor is not finite", fn);
  if (tokens == 0 || num_requests == 0) return ok();
  if ((s = mxq::check_rows(fn, "q", q, q_token_stride, q_head_stride, D)) != MXQ_OK) return s;
  if ((s = mxq::check_rows(fn, "q_out", q_out, out_token_stride, out_head_stride, D)) != MXQ_OK) return s;
  if ((s = mxq::check_rows(fn, "k", k, k_token_stride, k_head_stride, D)) != MXQ_OK) return s;
  if ((s = mxq::check_rows(fn, "v", v, v_token_stride, v_head_stride, D)) != MXQ_OK) return s;
  if (!inv_freq) return fail(MXQ_EINVAL, "%s: inv_freq is NULL", fn);
  if (!aligned(inv_freq, 4)) return fail(MXQ_EALIGN, "%s: inv_freq 4-byte aligned", fn);
  if (!aligned16(k_dq) || !aligned16(v_dq)) return fail(MXQ_EALIGN, "%s: k_dq and v_dq 16-byte aligned", fn);
  if (tokens >= (1 << 25)) return fail(MXQ_EUNSUPPORTED, "%s: too many rows for one call", fn);    // 32-bit grid
  a.p.k = k;
  a.p.v = v;
  a.p.T = tokens;
  a.p.k_token = k_token_stride;
  a.p.k_head = k_head_stride;
  a.p.v_token = v_token_stride;
  a.p.v_head = v_head_stride;
  a.p.k_dq = k_dq;
  a.p.v_dq = v_dq;
  a.q = q;
  a.Hq = num_q_heads;
  a.q_token = q_token_stride;
  a.q_head = q_head_stride;
  a.q_out = q_out;
  a.o_token = out_token_stride;
  a.o_head = out_head_stride;
  a.inv_freq = inv_freq;
  a.rot = rotary_dim;
  a.interleaved = interleaved != 0;
  a.factor = factor;
  return hip_status(mxq::launch_rope_append(a, S(stream)), fn);
}

}  // extern "C"
