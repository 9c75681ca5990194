// Host checks of a cache, a call's requests and its rows, shared by the entry
// points that write or read the paged NVFP4 cache.  Internal to the library.
#pragma once

#include "api_common.h"
#include "decode_kernels.h"
#include "mxq_decode.h"

namespace mxq {

constexpr int64_t I31 = (int64_t)1 << 31;

inline bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Fills c from the cache and the requests, or says what is wrong.
inline mxq_status cache_args(const char* fn, const mxq_cache* cache, const int32_t* block_table, int64_t ld_table,
                             int64_t table_width, const int32_t* seq_lens, const int32_t* q_offsets, int64_t num_requests,
                             int64_t tokens, CacheArgs* c) {
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
inline mxq_status check_rows(const char* fn, const char* name, const uint16_t* p, int64_t token, int64_t head, int D) {
  if (!p) return fail(MXQ_EINVAL, "%s: %s is NULL", fn, name);
  if (token < 0 || head < 0) return fail(MXQ_EINVAL, "%s: negative stride of %s", fn, name);
  if (!aligned16(p) || token % 8 || head % 8)
    return fail(MXQ_EALIGN, "%s: %s 16-byte aligned, its strides multiples of 8", fn, name);
  return MXQ_OK;
}

}  // namespace mxq
