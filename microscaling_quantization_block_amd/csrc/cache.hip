// New K and V rows into the pages of an NVFP4 cache.
//
// A row is the D values of one token and KV head.  It is quantized exactly as
// nvfp4_quantize does a row under a per-row second scale (nearest even):
// S = fl(amax / 2688), s_b = E4M3(fl(a_b / fl(6 S))), codes E2M1 of
// fl(x fl(1 / fl(s_b S))).  One with an infinity or a NaN gets a NaN for S:
// every value of it is NaN then, and the attention meets no infinite second scale,
// whose logits might be -infinity and look like tokens out of reach.
//
// D / 8 lanes hold a row, eight values each (one
// 16-byte load), a block is a lane pair; the row maximum is an integer
// maximum over the lanes.  A decode step (128 rows of 8 heads, 3.6 us) is one
// chain of latencies: request, offsets, page, store.  A prompt (10 k tokens of 8 heads)
// is bound by memory:
// 91 MB of rows, codes and dequantized rows in 30.1 us, 3.0 TB/s, where a large
// copy has 4.8; its rows are written as short pieces of many pages.
//
// V's block scales are stored [D / 16, P] inside a page (K's [P, D / 16]):
// the attention kernel contracts over tokens there and reads the scales of
// four neighbouring tokens of one block as one word.

#include "cache_device.h"
#include "nvfp4_device.h"

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

  const uint32_t m8 = amax8_bits(x);
  const uint32_t a_b = umax(m8, lane_xor_u32(m8, 1));
  uint32_t amax = a_b;
#pragma unroll
  for (int s = 2; s < L; s *= 2) amax = umax(amax, lane_xor_u32(amax, s));
  // a row with an infinity or a NaN: all its values are NaN
  const float S = amax < 0x7F800000u ? __uint_as_float(amax) / 2688.0f : __builtin_nanf("");
  const BlockScale bs = nv_block_scale(__uint_as_float(a_b), S);
  const u32x4 none = {0, 0, 0, 0};
  const uint32_t code = S < TINY_S ? nv_encode8<false, true>(x, bs.r, none) : nv_encode8<false, false>(x, bs.r, none);

  if (page >= 0) {
    const int P = 1 << c.P_log2;
    const int64_t slot = pos & (P - 1);
    const int64_t hs = h * P + slot;           // the row's index in the page
    uint8_t* codes = (is_v ? c.vc : c.kc) + page * c.pc + hs * (D / 2);
    *reinterpret_cast<uint32_t*>(codes + 4 * lane) = code;
    if ((lane & 1) == 0) {
      if (is_v) c.vs[page * c.psc + (h * (D / 16) + (lane >> 1)) * P + slot] = (uint8_t)bs.code;
      else c.ks[page * c.psc + hs * (D / 16) + (lane >> 1)] = (uint8_t)bs.code;
    }
    if (lane == 0) (is_v ? c.vg : c.kg)[page * c.pg + hs] = S;
  }
  uint16_t* dq = is_v ? a.v_dq : a.k_dq;
  if (dq) {
    // bf16(fl(fl(c s_b) S)), the dequantizer's chain
    const float sb = e4m3_to_f32(bs.code);
    mxq_f32x2 v[4];
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 0);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 1);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 2);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 3);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = f32x2_to_bf16x2((v[i].x * sb) * S, (v[i].y * sb) * S);
    *reinterpret_cast<uint4*>(dq + (t * c.H + h) * D + 8 * lane) = make_uint4(o[0], o[1], o[2], o[3]);
  }
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
