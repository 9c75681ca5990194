/*
 * mxq_decode.h -- the decode step of a 4-bit sampler: products of a few BF16
 * rows with NVFP4 weights, a paged K/V cache held in NVFP4, and attention over
 * that cache.  Included by mxq.h; the conventions there hold for every entry
 * (caller-owned device memory, work enqueued on the caller's stream, host
 * validation before any launch, no allocation, no exception).
 */
#ifndef MXQ_DECODE_H
#define MXQ_DECODE_H

#include "mxq.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * nvfp4_gemv -- y[m, n] = sum_k x[m, k] * dq(W)[n, k] for few rows m: BF16 x as
 * it is, NVFP4 weights, binary32 sums, one rounding to BF16.  For the rows of
 * a decode step (one to some tens per matrix): every 16 rows read the weights
 * once, so a prompt's rows are better quantized and given to mx_gemm.
 *   x, ld_x        BF16 [x_rows, K], row stride in elements
 *   w              NVFP4 operand [N, K] as mx_gemm takes for B: ROW or TILE
 *                  blocks, LINEAR or (ROW) MFMA scales, a per-tensor second
 *                  scale; not transposed.  Grouped: one matrix per group,
 *                  laid out as mx_gemm's grouped B.
 *   y, ld_y        BF16 [M, N]
 *   num_groups     0 for one matrix; else group_row_offsets [num_groups + 1]
 *                  (device int32, non-decreasing, within [0, M]): rows
 *                  [off[g], off[g+1]) use matrix g; rows of no group are
 *                  left as they were
 *   x_row_index    device int32 [M] or NULL: row m reads x row x_row_index[m];
 *                  an entry outside [0, x_rows) reads a row of zeros
 *   x_rows         rows of x (== M when x_row_index is NULL)
 * Sums run over x value(c) s_b, S multiplies them at the end: x below 2^100 in
 * magnitude (for K up to 2^16).
 * Shapes: K % 16 == 0; N % 16 == 0 (TILE), N % 32 == 0 and K % 64 == 0 (MFMA).
 * Alignment: x and the codes 16-byte aligned, ld_x % 8 == 0, w->ld % 16 == 0.
 */
mxq_status nvfp4_gemv(const uint16_t* x, int64_t ld_x, int64_t x_rows, const mxq_operand* w, int64_t M, int64_t N,
                      int64_t K, uint16_t* y, int64_t ld_y, int32_t num_groups, const int32_t* group_row_offsets,
                      const int32_t* x_row_index, void* stream);

/*
 * nvfp4_gemv_swiglu -- the gate_up product of a few rows with its SwiGLU:
 * h[m, i] = silu(g) * u, g = x[m] . W[i], u = x[m] . W[inter + i].  W has the gate
 * rows [0, inter), then the up rows (per group), as for mx_gemm_swiglu.  g and
 * u stay in binary32 (mx_gemm_swiglu rounds them to BF16 first).
 * Arguments as nvfp4_gemv with N = inter; the weight has 2 * inter rows.
 * TILE blocks need inter % 16 == 0, MFMA scales inter % 16 == 0.
 */
mxq_status nvfp4_gemv_swiglu(const uint16_t* x, int64_t ld_x, int64_t x_rows, const mxq_operand* w, int64_t M,
                             int64_t inter, int64_t K, uint16_t* h, int64_t ld_h, int32_t num_groups,
                             const int32_t* group_row_offsets, const int32_t* x_row_index, void* stream);

/*
 * A paged NVFP4 cache of K and V rows (a row: the head_dim values of one token
 * and KV head, quantized as nvfp4_quantize does a row of finite values, nearest
 * even, one second scale per row).  Inside a page everything is contiguous:
 *   k_codes, v_codes      [num_heads, page_size, head_dim / 2] bytes, low nibble even
 *   k_scales              [num_heads, page_size, head_dim / 16] E4M3
 *   v_scales              [num_heads, head_dim / 16, page_size] E4M3 (the
 *                         attention reads neighbouring tokens of a block)
 *   k_gscales, v_gscales  [num_heads, page_size] floats
 * and page p starts p * stride later: code_stride bytes, scale_stride bytes,
 * gscale_stride floats (at least a page; K and V pages may be interleaved).
 * head_dim 64, 128 or 256; page_size a power of two from 16 to 1024.
 * Alignment: codes and gscales 16 bytes, scales 4 bytes (strides alike).
 */
typedef struct {
  uint8_t* k_codes;
  uint8_t* k_scales;
  float* k_gscales;
  uint8_t* v_codes;
  uint8_t* v_scales;
  float* v_gscales;
  int64_t num_pages, code_stride, scale_stride, gscale_stride;
  int32_t num_heads, page_size, head_dim;
} mxq_cache;

/*
 * The requests of a call, all device int32:
 *   block_table [num_requests, table_width] (ld_table entries a row): page of
 *               each page_size positions of a request.  An entry outside
 *               [0, num_pages), or a position beyond the row, has no page: new
 *               rows there are not stored, and attention does not see them.
 *   seq_lens    [num_requests]: tokens of each request, the new ones included
 *   q_offsets   [num_requests + 1] or NULL: request b has the call's rows
 *               [q_offsets[b], q_offsets[b+1]), non-decreasing, within
 *               [0, tokens]; row i of them is position
 *               seq_lens[b] - (their number) + i.  NULL: one row per
 *               request (tokens == num_requests).  Rows before q_offsets[0] or
 *               from the last offset on belong to no request, and a request
 *               whose offsets leave [0, tokens] has no rows: nothing is read
 *               or written for either.
 *
 * nvfp4_cache_append -- quantizes the call's K and V rows into the cache.
 *   k, v             BF16 [tokens, num_heads, head_dim], strides in elements
 *                    (multiples of 8), head_dim contiguous, 16-byte aligned
 *   k_dq, v_dq       NULL, or BF16 [tokens, num_heads, head_dim] contiguous:
 *                    the values stored, bf16(fl(fl(c s_b) S)) as mx_dequantize
 *                    gives them (written also for a row without a page)
 * Two rows of one call that land on the same slot leave either of them there,
 * or a mixture.  A row with an infinity or a NaN is stored with a NaN second
 * scale, so that all its values are NaN.
 */
mxq_status nvfp4_cache_append(const uint16_t* k, int64_t k_token_stride, int64_t k_head_stride, const uint16_t* v,
                              int64_t v_token_stride, int64_t v_head_stride, int64_t tokens, const mxq_cache* cache,
                              const int32_t* block_table, int64_t ld_table, int64_t table_width,
                              const int32_t* seq_lens, const int32_t* q_offsets, int64_t num_requests,
                              uint16_t* k_dq, uint16_t* v_dq, void* stream);

/*
 * nvfp4_attention -- causal attention of the call's query rows over the cache:
 * row at position p, query head h: x_t = scale * q . dq(K_t) of KV head
 * h / (num_q_heads / num_heads), over t in (p - window, p] (window 0: [0, p]);
 * out = sum_t softmax(x)_t dq(V_t).  A row with nothing in reach (an empty
 * request, more rows than tokens, no pages) gives zeros and lse -infinity.
 * The rows' own K and V are read from the cache: append first.  Cache bytes
 * no row reaches may hold anything, and what one row reaches does not touch the
 * rows that do not.  A row becomes NaN by a NaN or an infinity in its q, by a NaN
 * in a K or V row that it reaches (a NaN among a token's V scales may spoil all of
 * that token's values), and by a largest x_t beyond binary32; its log sum too,
 * but for V.  Second scales are finite or NaN and not negative, as
 * nvfp4_cache_append stores them; K below 2^100 in magnitude.
 *   q, out       BF16 [tokens, num_q_heads, head_dim], strides in elements
 *                (multiples of 8), head_dim contiguous, 16-byte aligned
 *   lse          NULL, or binary32 [tokens, num_q_heads] contiguous: the natural
 *                log of sum_t exp(x_t)
 *   workspace    device, 16-byte aligned, nvfp4_attention_workspace() bytes (may
 *                be NULL if that is 0; a window may need less); its content
 *                before and after means nothing, calls in flight at once need one each
 * How the context is split follows from the shapes alone (table_width bounds
 * the lengths), so a captured call replays for any lengths, and equal calls
 * give equal bits.
 */
mxq_status nvfp4_attention(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, int64_t tokens,
                           int32_t num_q_heads, const mxq_cache* cache, const int32_t* block_table, int64_t ld_table,
                           int64_t table_width, const int32_t* seq_lens, const int32_t* q_offsets,
                           int64_t num_requests, float scale, int64_t window, uint16_t* out, int64_t out_token_stride,
                           int64_t out_head_stride, float* lse, void* workspace, int64_t workspace_bytes,
                           void* stream);
int64_t nvfp4_attention_workspace(int64_t tokens, int32_t num_q_heads, int32_t num_heads, int32_t head_dim,
                                  int32_t page_size, int64_t table_width, int64_t num_requests, int32_t ragged);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_DECODE_H */
