// C ABI of the decode step (include/mxq_decode.h): argument validation on the
// host, then kernel launches on the caller's stream, as in api.cpp.

#include <math.h>
#include <string.h>

#include "api_common.h"
#include "decode_kernels.h"
#include "mxq_decode.h"

using mxq::aligned16;
using mxq::fail;
using mxq::hip_status;
using mxq::ok;

namespace {

hipStream_t S(void* s) { return reinterpret_cast<hipStream_t>(s); }

constexpr int64_t I31 = (int64_t)1 << 31;

// An enumerator from the caller's memory as a plain number: a value the enum
// does not have must reach the checks, and loading it as the enum is undefined.
template <class E>
int number(const E& e) {
  int v;
  static_assert(sizeof(E) == sizeof(int), "C enums are ints");
  memcpy(&v, &e, sizeof(v));
  return v;
}

bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

mxq_status gemv_impl(const char* fn, const uint16_t* x, int64_t ld_x, int64_t x_rows, const mxq_operand* w, int64_t M,
                     int64_t N, int64_t K, uint16_t* y, int64_t ld_y, int32_t num_groups,
                     const int32_t* group_row_offsets, const int32_t* x_row_index, bool swiglu, void* stream) {
  if (!w) return fail(MXQ_EINVAL, "%s: null operand", fn);
  if (M < 0 || N < 0 || K < 0 || x_rows < 0 || num_groups < 0) return fail(MXQ_EINVAL, "%s: negative size", fn);
  const int fmt = number(w->fmt), block = number(w->block), gs = number(w->gs), layout = number(w->layout);
  if (fmt != MXQ_FMT_NVFP4) return fail(MXQ_EUNSUPPORTED, "%s: the weights must be NVFP4", fn);
  if (w->transposed) return fail(MXQ_EUNSUPPORTED, "%s: the weights must be row-major (not transposed)", fn);
  if (M == 0 || N == 0) return ok();
  if (K == 0) return fail(MXQ_EUNSUPPORTED, "%s: K == 0 (nothing would be written)", fn);
  if (!x || !y || !w->data || !w->scales || !w->gscales) return fail(MXQ_EINVAL, "%s: null pointer", fn);
  if (num_groups > 0 && !group_row_offsets) return fail(MXQ_EINVAL, "%s: grouped call without offsets", fn);
  if (!x_row_index && x_rows != M) return fail(MXQ_EINVAL, "%s: x_rows must equal M without a row index", fn);
  if (x_rows < 1) return fail(MXQ_EINVAL, "%s: x_rows < 1", fn);
  const int64_t wr = swiglu ? 2 * N : N;                       // rows of a matrix
  if (M >= I31 || N >= I31 / 64 || K >= I31 || num_groups > 65535)
    return fail(MXQ_EUNSUPPORTED, "%s: a size is too large (M, K < 2^31, N < 2^25, at most 65535 groups)", fn);
  if (K % 16) return fail(MXQ_ESHAPE, "%s: K %% 16 != 0 (K=%lld)", fn, (long long)K);
  if (gs != MXQ_GS_PER_TENSOR && gs != MXQ_GS_GIVEN)
    return fail(MXQ_EUNSUPPORTED, "%s: the weights take a per-tensor second scale", fn);
  mxq::GemvScales sl = mxq::GS_ROW;
  if (block == MXQ_BLOCK_TILE) {
    if (layout != MXQ_LAYOUT_LINEAR) return fail(MXQ_EUNSUPPORTED, "%s: the MFMA scale layout is for ROW blocks", fn);
    if (N % 16) return fail(MXQ_ESHAPE, "%s: tile blocks need rows %% 16 == 0 (N=%lld)", fn, (long long)N);
    sl = mxq::GS_TILE;
  } else if (block != MXQ_BLOCK_ROW) {
    return fail(MXQ_EINVAL, "%s: block must be ROW or TILE", fn);
  } else if (layout == MXQ_LAYOUT_MFMA) {
    if (wr % 32 || K % 64) return fail(MXQ_ESHAPE, "%s: MFMA scales need weight rows %% 32 == 0 and K %% 64 == 0", fn);
    sl = mxq::GS_MFMA;
  } else if (layout != MXQ_LAYOUT_LINEAR) {
    return fail(MXQ_EINVAL, "%s: bad scale layout", fn);
  }
  if (ld_x < K || w->ld < K || ld_y < N) return fail(MXQ_EINVAL, "%s: leading dimension smaller than the row", fn);
  if (!aligned16(x) || ld_x % 8 || !aligned16(w->data) || w->ld % 16 || !aligned(y, 2) || !aligned(w->gscales, 4))
    return fail(MXQ_EALIGN, "%s: x and the codes 16-byte aligned, ld_x %% 8 == 0, the weight's ld %% 16 == 0", fn);

  mxq::GemvArgs a = {};
  a.x = x;
  a.ld_x = ld_x;
  a.x_rows = x_rows;
  a.w = static_cast<const uint8_t*>(w->data);
  a.ld_w = w->ld / 2;
  a.w_group = wr * a.ld_w;
  a.scales = w->scales;
  a.s_group = (sl == mxq::GS_TILE ? wr / 16 : wr) * (K / 16);
  a.gs = w->gscales;
  a.M = M;
  a.N = N;
  a.K = K;
  a.y = y;
  a.ld_y = ld_y;
  a.num_groups = num_groups;
  a.offsets = group_row_offsets;
  a.row_index = x_row_index;
  return hip_status(mxq::launch_nvfp4_gemv(a, sl, swiglu, S(stream)), fn);
}

// Fills c from the cache and the requests, or says what is wrong.
mxq_status cache_args(const char* fn, const mxq_cache* cache, const int32_t* block_table, int64_t ld_table,
                      int64_t table_width, const int32_t* seq_lens, const int32_t* q_offsets, int64_t num_requests,
                      int64_t tokens, mxq::CacheArgs* c) {
  if (!cache) return fail(MXQ_EINVAL, "%s: cache is NULL", fn);
  if (tokens < 0 || num_requests < 0 || table_width < 0 || cache->num_pages < 0 || cache->num_heads < 0)
    return fail(MXQ_EINVAL, "%s: negative size", fn);
  const int D = cache->head_dim, P = cache->page_size;
  if (D != 64 && D != 128 && D != 256)
    return fail(MXQ_EUNSUPPORTED, "%s: head_dim must be 64, 128 or 256 (head_dim=%d)", fn, D);
  if (P < 16 || P > 1024 || (P & (P - 1)))
    return fail(MXQ_EUNSUPPORTED, "%s: page_size must be a power of two from 16 to 1024 (page_size=%d)", fn, P);
  if (cache->num_heads < 1 || cache->num_heads > 32767)
    return fail(MXQ_EINVAL, "%s: num_heads must be 1 to 32767", fn);
  if (!q_offsets && tokens != num_requests)
    return fail(MXQ_EINVAL, "%s: without q_offsets there is one row per request (tokens=%lld, requests=%lld)", fn,
                (long long)tokens, (long long)num_requests);
  if (tokens >= I31 || num_requests >= I31 || table_width > I31 / 2 / P || cache->num_pages >= I31)
    return fail(MXQ_EUNSUPPORTED, "%s: a size is too large (a table row covers at most 2^30 positions)", fn);
  if (tokens == 0 || num_requests == 0) return MXQ_OK;
  if (cache->num_pages < 1) return fail(MXQ_EINVAL, "%s: the cache has no pages", fn);
  if (!cache->k_codes || !cache->k_scales || !cache->k_gscales || !cache->v_codes || !cache->v_scales ||
      !cache->v_gscales || !seq_lens || (!block_table && table_width > 0))
    return fail(MXQ_EINVAL, "%s: null pointer", fn);
  if (ld_table < table_width) return fail(MXQ_EINVAL, "%s: ld_table < table_width", fn);
  const int64_t rows = (int64_t)cache->num_heads * P;
  if (cache->code_stride < rows * (D / 2) || cache->scale_stride < rows * (D / 16) || cache->gscale_stride < rows)
    return fail(MXQ_EINVAL, "%s: a page stride is smaller than a page", fn);
  if (cache->code_stride >= I31 || cache->scale_stride >= I31 || cache->gscale_stride >= I31 / 4)
    return fail(MXQ_EUNSUPPORTED, "%s: a page stride must be below 2 GiB", fn);
  if (!aligned16(cache->k_codes) || !aligned16(cache->v_codes) || !aligned16(cache->k_gscales) ||
      !aligned16(cache->v_gscales) || !aligned(cache->k_scales, 4) || !aligned(cache->v_scales, 4) ||
      cache->code_stride % 16 || cache->scale_stride % 4 || cache->gscale_stride % 4 || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(q_offsets, 4))
    return fail(MXQ_EALIGN, "%s: cache codes and second scales 16-byte, block scales 4-byte aligned, strides alike", fn);
  c->kc = cache->k_codes;
  c->ks = cache->k_scales;
  c->kg = cache->k_gscales;
  c->vc = cache->v_codes;
  c->vs = cache->v_scales;
  c->vg = cache->v_gscales;
  c->pages = cache->num_pages;
  c->pc = cache->code_stride;
  c->psc = cache->scale_stride;
  c->pg = cache->gscale_stride;
  c->H = cache->num_heads;
  c->D = D;
  c->P_log2 = __builtin_ctz((unsigned)P);
  c->table = block_table;
  c->ld_table = ld_table;
  c->width = table_width;
  c->seq_lens = seq_lens;
  c->q_offsets = q_offsets;
  c->B = num_requests;
  return MXQ_OK;
}

// [tokens, heads, D] rows of BF16 under two strides
mxq_status check_rows(const char* fn, const char* name, const uint16_t* p, int64_t token, int64_t head, int D) {
  if (!p) return fail(MXQ_EINVAL, "%s: %s is NULL", fn, name);
  if (token < 0 || head < 0) return fail(MXQ_EINVAL, "%s: negative stride of %s", fn, name);
  if (!aligned16(p) || token % 8 || head % 8)
    return fail(MXQ_EALIGN, "%s: %s 16-byte aligned, its strides multiples of 8", fn, name);
  return MXQ_OK;
}

}  // namespace

extern "C" {

mxq_status nvfp4_gemv(const uint16_t* x, int64_t ld_x, int64_t x_rows, const mxq_operand* w, int64_t M, int64_t N,
                      int64_t K, uint16_t* y, int64_t ld_y, int32_t num_groups, const int32_t* group_row_offsets,
                      const int32_t* x_row_index, void* stream) {
  return gemv_impl("nvfp4_gemv", x, ld_x, x_rows, w, M, N, K, y, ld_y, num_groups, group_row_offsets, x_row_index,
                   false, stream);
}

mxq_status nvfp4_gemv_swiglu(const uint16_t* x, int64_t ld_x, int64_t x_rows, const mxq_operand* w, int64_t M,
                             int64_t inter, int64_t K, uint16_t* h, int64_t ld_h, int32_t num_groups,
                             const int32_t* group_row_offsets, const int32_t* x_row_index, void* stream) {
  return gemv_impl("nvfp4_gemv_swiglu", x, ld_x, x_rows, w, M, inter, K, h, ld_h, num_groups, group_row_offsets,
                   x_row_index, true, stream);
}

mxq_status nvfp4_cache_append(const uint16_t* k, int64_t k_token_stride, int64_t k_head_stride, const uint16_t* v,
                              int64_t v_token_stride, int64_t v_head_stride, int64_t tokens, const mxq_cache* cache,
                              const int32_t* block_table, int64_t ld_table, int64_t table_width,
                              const int32_t* seq_lens, const int32_t* q_offsets, int64_t num_requests,
                              uint16_t* k_dq, uint16_t* v_dq, void* stream) {
  const char* fn = "nvfp4_cache_append";
  mxq::AppendArgs a = {};
  mxq_status s = cache_args(fn, cache, block_table, ld_table, table_width, seq_lens, q_offsets, num_requests, tokens,
                            &a.c);
  if (s != MXQ_OK) return s;
  if (tokens == 0 || num_requests == 0) return ok();
  const int D = cache->head_dim;
  if ((s = check_rows(fn, "k", k, k_token_stride, k_head_stride, D)) != MXQ_OK) return s;
  if ((s = check_rows(fn, "v", v, v_token_stride, v_head_stride, D)) != MXQ_OK) return s;
  if (!aligned16(k_dq) || !aligned16(v_dq)) return fail(MXQ_EALIGN, "%s: k_dq and v_dq 16-byte aligned", fn);
  const int64_t wg_rows = 2048 / D;            // a workgroup's; its 256 lanes times the grid stay below 2^32
  if ((tokens + wg_rows - 1) / wg_rows * 2 * cache->num_heads >= I31 / 128)
    return fail(MXQ_EUNSUPPORTED, "%s: too many rows for one call", fn);
  a.k = k;
  a.v = v;
  a.T = tokens;
  a.k_token = k_token_stride;
  a.k_head = k_head_stride;
  a.v_token = v_token_stride;
  a.v_head = v_head_stride;
  a.k_dq = k_dq;
  a.v_dq = v_dq;
  return hip_status(mxq::launch_cache_append(a, S(stream)), fn);
}

int64_t nvfp4_attention_workspace(int64_t tokens, int32_t num_q_heads, int32_t num_heads, int32_t head_dim,
                                  int32_t page_size, int64_t table_width, int64_t num_requests, int32_t ragged) {
  if (tokens <= 0 || num_requests <= 0 || num_heads <= 0 || num_q_heads < num_heads || head_dim <= 0) return 0;
  if (tokens >= I31 || num_requests >= I31 || page_size <= 0 || table_width < 0 || table_width > I31 / 2 / page_size)
    return 0;                                  // nvfp4_attention refuses these
  const mxq::AttnPlan p = mxq::plan_attention(num_requests, tokens, num_heads, num_q_heads / num_heads, head_dim,
                                              table_width * page_size, ragged != 0);
  return mxq::attention_workspace(p, num_requests, num_heads, head_dim);
}

mxq_status nvfp4_attention(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, int64_t tokens,
                           int32_t num_q_heads, const mxq_cache* cache, const int32_t* block_table, int64_t ld_table,
                           int64_t table_width, const int32_t* seq_lens, const int32_t* q_offsets,
                           int64_t num_requests, float scale, int64_t window, uint16_t* out, int64_t out_token_stride,
                           int64_t out_head_stride, float* lse, void* workspace, int64_t workspace_bytes,
                           void* stream) {
  const char* fn = "nvfp4_attention";
  mxq::AttnArgs a = {};
  mxq_status s = cache_args(fn, cache, block_table, ld_table, table_width, seq_lens, q_offsets, num_requests, tokens,
                            &a.c);
  if (s != MXQ_OK) return s;
  const int D = cache->head_dim, H = cache->num_heads;
  if (num_q_heads < 1 || num_q_heads % H)
    return fail(MXQ_ESHAPE, "%s: num_q_heads must be a multiple of the cache's heads (%d, %d)", fn, num_q_heads, H);
  if (window < 0) return fail(MXQ_EINVAL, "%s: negative window", fn);
  if (!isfinite(scale)) return fail(MXQ_EINVAL, "%s: scale is not finite", fn);
  if (tokens == 0 || num_requests == 0) return ok();
  if ((s = check_rows(fn, "q", q, q_token_stride, q_head_stride, D)) != MXQ_OK) return s;
  if ((s = check_rows(fn, "out", out, out_token_stride, out_head_stride, D)) != MXQ_OK) return s;
  if (!aligned(lse, 4)) return fail(MXQ_EALIGN, "%s: lse 4-byte aligned", fn);
  a.window = window < I31 ? window : 0;        // positions lie below 2^31: it holds them all
  // no row sees more than this
  const int64_t capacity = table_width * cache->page_size;
  const int64_t reach = a.window && a.window + tokens < capacity ? a.window + tokens : capacity;
  const mxq::AttnPlan p = mxq::plan_attention(num_requests, tokens, H, num_q_heads / H, D, reach, q_offsets != nullptr);
  if (p.units * H >= I31 / 256 || tokens * num_q_heads >= I31 / 32)      // 32-bit grids
    return fail(MXQ_EUNSUPPORTED, "%s: too many rows for one call", fn);
  const int64_t need = mxq::attention_workspace(p, num_requests, H, D);
  if (need) {
    if (!workspace || workspace_bytes < need)
      return fail(MXQ_EINVAL, "%s: the workspace needs %lld bytes", fn, (long long)need);
    if (!aligned16(workspace)) return fail(MXQ_EALIGN, "%s: workspace 16-byte aligned", fn);
  }
  a.q = q;
  a.T = tokens;
  a.q_token = q_token_stride;
  a.q_head = q_head_stride;
  a.Hq = num_q_heads;
  a.G = num_q_heads / H;
  a.scale_log2 = scale * 1.44269504088896340736f;
  a.out = out;
  a.o_token = out_token_stride;
  a.o_head = out_head_stride;
  a.lse = lse;
  a.target = p.target;
  a.coarse = p.coarse;
  a.units = p.units;
  if (need) {
    const int64_t rows = p.units * H * p.ct;
    a.part_o = static_cast<float*>(workspace);
    a.part_index = reinterpret_cast<int2*>(a.part_o + rows * D);
    a.part_lse = reinterpret_cast<float*>(a.part_index + num_requests);
  }
  return hip_status(mxq::launch_attention(a, p, S(stream)), fn);
}

}  // extern "C"
