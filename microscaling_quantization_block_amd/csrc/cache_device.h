// Addressing of the paged NVFP4 cache shared by the kernels that write and
// read it, and the row that the appending kernels store.
#pragma once

#include "decode_kernels.h"
#include "nvfp4_device.h"
#include "requests.h"

namespace mxq {

// The page of cache position pos of request b, or -1: a position outside the
// table's row, or an entry outside [0, pages).
__device__ __forceinline__ int64_t page_of(const CacheArgs& c, int64_t b, int64_t pos) {
  const int64_t i = pos >> c.P_log2;
  if (pos < 0 || i >= c.width) return -1;
  const int64_t p = c.table[b * c.ld_table + i];
  return p < c.pages ? p : -1;                 // negative entries pass through
}

// Quantizes one row (the D values of one token and KV head h; D / 8
// neighbouring lanes hold eight values each, `lane` of them) and stores it at
// position pos in `page` (negative: nowhere), its values to dq_row where that is given.
//
// A row is quantized exactly as nvfp4_quantize does a row under a per-row
// second scale (nearest even): S = fl(amax / 2688), s_b = E4M3(fl(a_b / fl(6 S))),
// codes E2M1 of fl(x fl(1 / fl(s_b S))); a block is a lane pair, the row maximum
// an integer maximum over the lanes.  One with an infinity or a NaN gets a NaN
// for S: every value of it is NaN then, and the attention meets no infinite second
// scale, whose logits might be -infinity and look like tokens out of reach.
//
// V's block scales are stored [D / 16, P] inside a page (K's [P, D / 16]):
// the attention kernel contracts over tokens there and reads the scales of
// four neighbouring tokens of one block as one word.
template <int D>
__device__ __forceinline__ void append_row(const CacheArgs& c, bool is_v, int64_t h, int64_t page, int64_t pos,
                                           int lane, uint4 x, uint16_t* dq_row) {
  constexpr int L = D / 8;                     // lanes of a row
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
  if (dq_row) {
    // bf16(fl(fl(c s_b) S)), the dequantizer's chain
    *reinterpret_cast<uint4*>(dq_row + 8 * lane) = nv_decode8(code, e4m3_to_f32(bs.code), S);
  }
}

}  // namespace mxq
