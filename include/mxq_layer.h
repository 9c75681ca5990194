/*
 * mxq_layer.h -- the steps of a decoder layer around its quantized products:
 * the root-mean-square norm with the residual's addition and a quantized
 * output, and its gradient.
 * Included by mxq.h; the conventions there hold for every entry (caller-owned
 * device memory, work enqueued on the caller's stream, host validation before
 * any launch, no allocation, no exception).
 */
#ifndef MXQ_LAYER_H
#define MXQ_LAYER_H

#include "mxq.h"
#include "mxq_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * mx_rmsnorm -- for every row (token) of x [rows, cols]:
 *   h    = bf16(x + residual)                       (x without a residual)
 *   rstd = fl(1 / sqrt(mean(h^2) + eps))            (the mean in binary64)
 *   y    = bf16(fl(fl(h rstd) weight))
 * and, with fmt other than MXQ_FMT_BF16, the rowwise quantized copy of y that
 * the next product reads, with the bytes the quantizers give for y (the two
 * paths share their code): MXFP8 as mx_quantize(ROW), NVFP4 as
 * nvfp4_quantize(ROW, PER_ROW, RNE), FP8_B128 and FP8_B128_F32 as
 * fp8bw_quantize and fp8bw_quantize_f32 (ROW).
 * A row's outputs have the same bits whatever the number of rows.
 *   x, residual     BF16, row strides ld_x, ld_r (elements); residual may be NULL
 *   weight          BF16 [cols]
 *   h, ld_h         BF16 or NULL; only with a residual (may be x or residual
 *                   itself, with its stride)
 *   y, ld_y         BF16 or NULL (needed with MXQ_FMT_BF16); may be x itself
 *                   where h is not
 *   rstd            binary32 [rows] or NULL: what mx_rmsnorm_backward takes
 *   codes, ld_codes the codes, row stride in bytes (NULL with MXQ_FMT_BF16)
 *   scales          block scales, bytes (FP8_B128_F32: floats); `layout` MFMA is
 *                   for MXFP8 and NVFP4
 *   gscales         NVFP4: binary32 [rows]
 *   dq, ld_dq       BF16 or NULL: the values the codes stand for, as
 *                   mx_dequantize gives them (not with MXQ_FMT_BF16)
 * Shapes: cols % 8 == 0, the format's block divides cols; cols up to 32768.
 * MFMA scales: rows % 32 == 0, cols a multiple of four blocks.
 * Alignment: 16 bytes, strides multiples of 16 bytes; rstd and gscales 4 bytes.
 * A row with an infinity or a NaN, or with eps 0 and nothing but zeros, becomes
 * NaN (or 0 where a finite value meets an infinite sum); its codes and scales are then unspecified.
 */
mxq_status mx_rmsnorm(const uint16_t* x, int64_t ld_x, const uint16_t* residual, int64_t ld_r,
                      const uint16_t* weight, int64_t rows, int64_t cols, float eps, uint16_t* h, int64_t ld_h,
                      uint16_t* y, int64_t ld_y, float* rstd, mxq_format fmt, mxq_scale_layout layout,
                      uint8_t* codes, int64_t ld_codes, void* scales, float* gscales, uint16_t* dq, int64_t ld_dq,
                      void* stream);

/*
 * mx_rmsnorm_backward -- the gradient of y = h rstd(h) weight:
 *   dx[r] = rstd (g - xhat mean(g xhat)) + dresidual,  g = dy weight,  xhat = h rstd
 *   dweight = sum over rows of dy xhat
 * in binary32, dx rounded to BF16 once.  dx is the gradient of x and of the residual alike.
 *   dy, h, dresidual  BF16 [rows, cols]; h as mx_rmsnorm wrote it (x without a
 *                     residual); dresidual may be NULL: the gradient that reaches h
 *                     by the residual stream
 *   rstd              binary32 [rows] of mx_rmsnorm
 *   dx, ld_dx         BF16; may be dy or dresidual itself, with its stride
 *   dweight           binary32 [cols] or NULL
 *   workspace         device, 16-byte aligned, mx_rmsnorm_backward_workspace()
 *                     bytes (may be NULL where dweight is); calls in flight at once need one each
 * rows == 0 gives a dweight of zeros.  Equal calls give equal bits.
 * Shapes and alignment as mx_rmsnorm (cols % 8 == 0).
 */
mxq_status mx_rmsnorm_backward(const uint16_t* dy, int64_t ld_dy, const uint16_t* h, int64_t ld_h,
                               const uint16_t* weight, const float* rstd, const uint16_t* dresidual,
                               int64_t ld_dr, int64_t rows, int64_t cols, uint16_t* dx, int64_t ld_dx,
                               float* dweight, void* workspace, int64_t workspace_bytes, void* stream);
int64_t mx_rmsnorm_backward_workspace(int64_t rows, int64_t cols);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_LAYER_H */
