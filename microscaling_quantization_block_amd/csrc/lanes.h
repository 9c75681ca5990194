// Sums and maxima over 16 neighbouring lanes or a whole wave.
#pragma once

#include "mxq_device.h"

namespace mxq {

// v of another lane of the same 16 by a DPP control
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
__device__ __forceinline__ double read_f64(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ float read_f32(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}

// Sums and maxima over 16 lanes or a whole wave: quad permutes, half-row and row
// mirrors (a binary tree over lane numbers), then the four rows of 16.
template <int LANES>
__device__ __forceinline__ double lanes_sum(double v) {
  v += dpp_f64<0xB1>(v);
  v += dpp_f64<0x4E>(v);
  v += dpp_f64<0x141>(v);
  v += dpp_f64<0x140>(v);
  if constexpr (LANES == 16) return v;
  return (read_f64(v, 0) + read_f64(v, 16)) + (read_f64(v, 32) + read_f64(v, 48));
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  v += dpp_f32<0xB1>(v);
  v += dpp_f32<0x4E>(v);
  v += dpp_f32<0x141>(v);
  v += dpp_f32<0x140>(v);
  if constexpr (LANES == 16) return v;
  return (read_f32(v, 0) + read_f32(v, 16)) + (read_f32(v, 32) + read_f32(v, 48));
}
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  if constexpr (LANES == 64) return wave_max_u32(v);
  v = umax(v, dpp_u32<0xB1>(v));
  v = umax(v, dpp_u32<0x4E>(v));
  v = umax(v, dpp_u32<0x141>(v));
  return umax(v, dpp_u32<0x140>(v));
}

}  // namespace mxq
