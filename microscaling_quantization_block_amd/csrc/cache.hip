// New K and V rows into the pages of an NVFP4 cache.
//
// D / 8 lanes hold a row, eight values each (one 16-byte load); what they store
// is append_row's (cache_device.h).  A decode step (128 rows of 8 heads, 3.6 us) is one
// chain of latencies: request, offsets, page, store.  A prompt (10 k tokens of 8 heads)
// is bound by memory:
// 91 MB of rows, codes and dequantized rows in 30.1 us, 3.0 TB/s, where a large
// copy has 4.8; its rows are written as short pieces of many pages.

#include "cache_device.h"

namespace mxq {

template <int D>
__global__ __launch_bounds__(256) void cache_append_kernel(AppendArgs a) {
  constexpr int L = D / 8;                     // lanes of a row
  const CacheArgs& c = a.c;
  // Neighbouring workgroups hold neighbouring heads of the same tokens: together
  // they read whole tokens.  The values are loaded before the request and the page
  // are looked up, which do not need them.  (The tokens of one head first and the
  // values after the request: 32.3 us against 29.7 for the prompt above; only
  // this order of workgroups: 32.4.  Four rows per lane group: 32.2.)
  const int hv = blockIdx.x % (2 * c.H);       // K's heads, then V's
  const int64_t t = (int64_t)(blockIdx.x / (2 * c.H)) * (256 / L) + threadIdx.x / L;
  const int lane = threadIdx.x & (L - 1);
  if (t >= a.T) return;                        // whole rows leave: the lane exchanges below stay inside a row
  const bool is_v = hv >= c.H;
  const int64_t h = is_v ? hv - c.H : hv;
  const uint16_t* src = is_v ? a.v + t * a.v_token + h * a.v_head : a.k + t * a.k_token + h * a.k_head;
  const uint4 x = *reinterpret_cast<const uint4*>(src + 8 * lane);
  RequestRows rows;
  const int64_t b = request_of(c, t, a.T, rows);
  if (b < 0) return;
  const int64_t pos = (int64_t)c.seq_lens[b] - rows.len + (t - rows.begin);
  const int64_t page = page_of(c, b, pos);

  uint16_t* dq = is_v ? a.v_dq : a.k_dq;
  append_row<D>(c, is_v, h, page, pos, lane, x, dq ? dq + (t * c.H + h) * D : nullptr);
}

hipError_t launch_cache_append(const AppendArgs& a, hipStream_t st) {
  const int64_t rows = 256 / (a.c.D / 8);      // of a workgroup
  const dim3 grid((unsigned)((a.T + rows - 1) / rows * 2 * a.c.H));
  if (a.c.D == 64) hipLaunchKernelGGL(cache_append_kernel<64>, grid, dim3(256), 0, st, a);
  else if (a.c.D == 128) hipLaunchKernelGGL(cache_append_kernel<128>, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(cache_append_kernel<256>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace mxq
