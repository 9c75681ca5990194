// FP8 element chains shared by the quantizers and by the norm that quantizes its
// output (the same code, so the same bits): block scales from a block's amax
// (power of two or binary32) and the 8-value encoders.
#pragma once

#include "mxq_device.h"

namespace mxq {

__device__ __forceinline__ uint32_t e8m0_from_amax_bits(uint32_t amax16) {
  int E = (int)(amax16 >> 7);
  int M = (int)(amax16 & 0x7F);
  int code = E - 8 + (M > 96 ? 1 : 0);
  return (uint32_t)(code < 0 ? 0 : code);
}

// Encode 8 BF16 values (in 4 words) with block exponent code s (e = s - 127):
// returns 8 E4M3 bytes in two words.
__device__ __forceinline__ uint2 mx_encode8(uint4 v, uint32_t s) {
  int sh = 127 - (int)s;   // multiply by 2^-e
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = __builtin_ldexpf(bf16_lo(w[i]), sh);
    float b = __builtin_ldexpf(bf16_hi(w[i]), sh);
    o[i] = f32x2_to_e4m3(a, b);
  }
  return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}

__device__ __forceinline__ uint32_t absmax8(uint4 v) {
  return umax(umax(bf16x2_absmax_bits(v.x), bf16x2_absmax_bits(v.y)),
              umax(bf16x2_absmax_bits(v.z), bf16x2_absmax_bits(v.w)));
}

// Blockwise FP8 with binary32 scales (F32S): s = amax / 448 (one correctly
// rounded division), codes E4M3 RNE of the binary32 quotient x / s clamped to
// +-448 (the quotient of the block maximum may exceed 448 by an ulp); a zero
// block stores s = 0 and zero codes.  A scale travels as its binary32 bits in
// the same uint32_t that carries an E8M0 code otherwise.
__device__ __forceinline__ uint32_t f32s_from_amax_bits(uint32_t amax16) {
  return __float_as_uint(__uint_as_float(amax16 << 16) / 448.0f);
}

// The quotient without a division per element: with r = RN(1/s) (one
// correctly rounded division per block), q0 = RN(x r), the exact residual
// x - q0 s by one FMA and the corrected q0 + residual * r by another.  The
// result can differ from RN(x / s) in its last bits, but for every BF16 x in
// a block and every scale s >= 2^-80 of a BF16 block maximum it gives the
// same E4M3 code (an exhaustive check over all 1.0e9 such pairs is among the
// host tests); smaller scales divide directly.
// (The sign is x's: for x = -0 the corrected sum would come out +0.)
__device__ __forceinline__ float f32s_quotient(float x, float sc, float r) {
  const float q0 = x * r;
  return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q0, sc, x), r, q0), x);
}

__device__ __forceinline__ uint2 f32s_encode8(uint4 v, uint32_t sbits) {
  const float sc = __uint_as_float(sbits);
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float q[8];
  if (sbits == 0u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = 0.0f;
  } else if (sc < 0x1p-80f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[2 * i] = bf16_lo(w[i]) / sc;
      q[2 * i + 1] = bf16_hi(w[i]) / sc;
    }
  } else {
    const float r = 1.0f / sc;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[2 * i] = f32s_quotient(bf16_lo(w[i]), sc, r);
      q[2 * i + 1] = f32s_quotient(bf16_hi(w[i]), sc, r);
    }
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = f32x2_to_e4m3(fminf(fmaxf(q[2 * i], -448.0f), 448.0f), fminf(fmaxf(q[2 * i + 1], -448.0f), 448.0f));
  return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}

template <bool F32S>
__device__ __forceinline__ uint32_t blk_scale(uint32_t amax16) {
  if constexpr (F32S) return f32s_from_amax_bits(amax16);
  return e8m0_from_amax_bits(amax16);
}

template <bool F32S>
__device__ __forceinline__ uint2 blk_encode8(uint4 v, uint32_t s) {
  if constexpr (F32S) return f32s_encode8(v, s);
  return mx_encode8(v, s);
}

// store scale s at element index i of a byte (E8M0) or binary32 scale array
template <bool F32S>
__device__ __forceinline__ void blk_store(uint8_t* scales, int64_t i, uint32_t s) {
  if constexpr (F32S) reinterpret_cast<float*>(scales)[i] = __uint_as_float(s);
  else scales[i] = (uint8_t)s;
}

}  // namespace mxq
