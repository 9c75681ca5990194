/*
 * mxq_layer.h -- the steps of a decoder layer around its quantized products:
 * the root-mean-square norm with the residual's addition and a quantized
 * output, the router of a layer with experts, the rows of its tokens ordered by
 * expert and back, each with its gradient; rotary positions on the way into the
 * NVFP4 cache.
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
 * Alignment: 16 bytes, strides multiples of 16 bytes (NVFP4 codes: of 8); rstd
 * and gscales 4 bytes.
 * A row with an infinity or a NaN, or with eps 0 and nothing but zeros, becomes
 * NaN (or 0 where a finite value meets an infinite sum); with eps 0, a row whose
 * rstd is beyond binary32 becomes infinite.  Codes and scales of such a row are unspecified.
 */
mxq_status mx_rmsnorm(const uint16_t* x, int64_t ld_x, const uint16_t* residual, int64_t ld_r,
                      const uint16_t* weight, int64_t rows, int64_t cols, double eps, uint16_t* h, int64_t ld_h,
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

/*
 * The rows of a layer with experts.  Token t uses the experts
 * experts[t, 0 .. topk - 1]; each such slot has one row in the experts' products,
 * and the rows are ordered by (expert, token, slot):
 *   offsets    [num_experts + 1]: expert e has the rows [offsets[e], offsets[e+1])
 *              (group_row_offsets of mx_gemm, mx_gemm_swiglu, nvfp4_gemv ...)
 *   row_token  [tokens * topk]: the token of every row (a_row_index, x_row_index);
 *              0 from row offsets[num_experts] on, rows that no expert has
 *   row_of     [tokens, topk]: the row of every slot, -1 for a slot without one
 * A slot whose expert is outside [0, num_experts) has no row: experts that are on
 * another device, or none.
 *
 * mx_moe_sort -- these three from given ids, experts int32 [tokens, topk].
 *
 * mx_moe_route -- the router: experts[t] are the topk largest logits of token t,
 * largest first, ties to the lower expert, and weights[t] their softmax
 * probabilities: over the chosen experts (renormalize) or over all of them.  An
 * expert whose logit is -infinity is never chosen: its slot has the id -1, the weight 0 and no
 * row.  A NaN counts as the largest logit, and makes its token's weights NaN,
 * as an infinity does.  Then the rows as mx_moe_sort orders them.
 *   logits       binary32 (logits_f32) or BF16 [tokens, num_experts], row stride ld
 *   experts      int32 [tokens, topk], weights binary32 [tokens, topk]: outputs
 *   workspace    device, 16-byte aligned, mx_moe_workspace() bytes (may be NULL if
 *                that is 0); calls in flight at once need one each
 *
 * mx_moe_route_backward -- dlogits [tokens, num_experts] (type of the logits, row stride ld_d)
 * from dweights [tokens, topk] and what mx_moe_route gave; the choice itself
 * has no gradient.
 *
 * Sizes: num_experts up to 1024, topk up to 64 and num_experts; tokens below
 * 2^24, tokens * topk at most 2^26 - 4.  tokens == 0 gives offsets of zeros.
 */
mxq_status mx_moe_route(const void* logits, int32_t logits_f32, int64_t ld, int64_t tokens, int32_t num_experts,
                        int32_t topk, int32_t renormalize, int32_t* experts, float* weights, int32_t* offsets,
                        int32_t* row_token, int32_t* row_of, void* workspace, int64_t workspace_bytes, void* stream);
mxq_status mx_moe_route_backward(const float* dweights, const void* logits, int32_t logits_f32, int64_t ld,
                                 int64_t tokens, int32_t num_experts, int32_t topk, int32_t renormalize,
                                 const int32_t* experts, const float* weights, void* dlogits, int64_t ld_d,
                                 void* stream);
mxq_status mx_moe_sort(const int32_t* experts, int64_t tokens, int32_t num_experts, int32_t topk, int32_t* offsets,
                       int32_t* row_token, int32_t* row_of, void* workspace, int64_t workspace_bytes, void* stream);
int64_t mx_moe_workspace(int64_t tokens, int32_t num_experts, int32_t topk);

/*
 * Tokens to the experts' rows and back, by row_of int32 [tokens, topk].  An entry
 * outside [0, num_rows) has no row: nothing is read or written for it.  Rows that no
 * entry names are left as they were.  Each row belongs to one entry (as
 * mx_moe_sort makes them); where two entries of mx_moe_dispatch or
 * mx_moe_combine_backward name one row, either is left there, or a mixture.
 *
 * mx_moe_dispatch -- rows[row_of[t, j]] = x[t], BF16.  (The products gather by row_token
 * themselves; this is for what needs the rows in memory: a BF16 or rowwise
 * quantized operand, products of one expert's rows at a time.  Experts' ranges start
 * at any row, so a block of 16 rows or more of a columnwise or tile copy may hold rows of two
 * experts: such a copy is no operand of a weight gradient per expert.)  Its gradient is
 * mx_moe_combine of the rows' gradients with weights NULL.
 *
 * mx_moe_combine -- out[t] = sum over j of weights[t, j] rows[row_of[t, j]], in
 * binary32 in the order of j, one rounding to BF16; weights NULL: ones.  A token
 * without rows gives zeros.
 *
 * mx_moe_combine_backward -- the gradient of mx_moe_combine:
 *   drows[row_of[t, j]] = weights[t, j] dout[t]      (BF16)
 *   dweights[t, j]      = dout[t] . rows[row_of[t, j]]  (binary32; 0 without a row)
 *
 * Matrices are BF16 with row strides in elements; cols % 8 == 0, 16-byte
 * alignment, strides multiples of 8.  Sizes as mx_moe_sort; cols below 2^26.
 */
mxq_status mx_moe_dispatch(const uint16_t* x, int64_t ld_x, int64_t tokens, int64_t cols, const int32_t* row_of,
                           int32_t topk, uint16_t* rows, int64_t ld_rows, int64_t num_rows, void* stream);
mxq_status mx_moe_combine(const uint16_t* rows, int64_t ld_rows, int64_t num_rows, const int32_t* row_of,
                          const float* weights, int64_t tokens, int64_t cols, int32_t topk, uint16_t* out,
                          int64_t ld_out, void* stream);
mxq_status mx_moe_combine_backward(const uint16_t* dout, int64_t ld_dout, const uint16_t* rows, int64_t ld_rows,
                                   int64_t num_rows, const int32_t* row_of, const float* weights, int64_t tokens,
                                   int64_t cols, int32_t topk, uint16_t* drows, int64_t ld_drows, float* dweights,
                                   void* stream);

/*
 * nvfp4_rope_append -- rotary positions for the call's rows q and k, and k and
 * v quantized into the cache as nvfp4_cache_append does it.  The requests, the
 * cache, k, v, k_dq and v_dq are those of nvfp4_cache_append; a row at position
 * p (seq_lens[b] - rows + i, as there) has the first rotary_dim values of every q
 * and k head turned by the angles p inv_freq[i], i < rotary_dim / 2:
 *   (a, b) -> (a c - b s, b c + a s),  c = fl(factor cos), s = fl(factor sin)
 * where (a, b) are the values (i, i + rotary_dim / 2), or (2 i, 2 i + 1) with
 * `interleaved`.  Cosine and sine are taken in binary64, the products and their
 * sum in binary32, and the turned row is rounded to BF16: q_out gets it, and the
 * cache the bytes of nvfp4_cache_append for the turned k.  Positions scaled for
 * long contexts are other frequencies (and a factor).
 *   q, q_out      BF16 [tokens, num_q_heads, head_dim], strides in elements
 *                 (multiples of 8), head_dim contiguous, 16-byte aligned; q_out
 *                 may be q itself, with its strides.  Rows of no request are not written.
 *   inv_freq      binary32 [rotary_dim / 2], on the device; p inv_freq[i] below 2^40
 *   rotary_dim    a multiple of 16, up to head_dim
 * Any num_q_heads from 1 to 32767: q and the cache need not belong to one attention.
 * tokens below 2^25.
 */
mxq_status nvfp4_rope_append(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, int32_t num_q_heads,
                             const uint16_t* k, int64_t k_token_stride, int64_t k_head_stride, const uint16_t* v,
                             int64_t v_token_stride, int64_t v_head_stride, int64_t tokens, const mxq_cache* cache,
                             const int32_t* block_table, int64_t ld_table, int64_t table_width,
                             const int32_t* seq_lens, const int32_t* q_offsets, int64_t num_requests,
                             const float* inv_freq, int32_t rotary_dim, int32_t interleaved, double factor,
                             uint16_t* q_out, int64_t out_token_stride, int64_t out_head_stride, uint16_t* k_dq,
                             uint16_t* v_dq, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_LAYER_H */
