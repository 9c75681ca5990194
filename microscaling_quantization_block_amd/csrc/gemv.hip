// Few BF16 rows times NVFP4 weights: y[m, n] = sum_k x[m, k] value(c) s_b S.
//
// The products are exact: an E2M1 code times its E4M3 block scale has at most
// six significant bits and lies in 2^-10 .. 2688, so it is a BF16 number, and
// the BF16 matrix instruction multiplies it with x unrounded and sums in
// binary32.  S leaves the sum and multiplies it once, in binary32; one
// rounding to BF16 ends the chain.
//
// One workgroup owns 16 weight rows (with SwiGLU 16 gate rows and their up
// rows) and all of K; its waves take 128-wide K chunks in turn and their
// partial tiles meet in LDS, so there are many loads in flight for a
// matrix with few rows and no second launch.  The weights are the left
// operand: lane (r, g) = (lane % 16, lane / 16) reads 16 bytes, the codes
// k0 + 32 g .. + 31 of row r, and feeds them to four matrix instructions
// eight at a time; x is read in the same order, so k is permuted alike on
// both sides and nothing is shuffled.

#include "mxq_device.h"
#include "decode_kernels.h"

namespace mxq {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Eight codes (one dword) times their block scale, as BF16 (exact).
__device__ __forceinline__ bf16x8 e2m1x8_to_bf16(uint32_t w, float s) {
  const mxq_f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
  const mxq_f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  const mxq_f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
  const mxq_f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  uint4 o;
  o.x = f32x2_to_bf16x2(a.x * s, a.y * s);
  o.y = f32x2_to_bf16x2(b.x * s, b.y * s);
  o.z = f32x2_to_bf16x2(c.x * s, c.y * s);
  o.w = f32x2_to_bf16x2(d.x * s, d.y * s);
  return __builtin_bit_cast(bf16x8, o);
}

// Byte offset of the scale of (row, block b) in one matrix of B blocks a row.
template <int SL>
__device__ __forceinline__ int64_t gemv_scale_offset(int64_t row, int64_t b, int64_t B) {
  if (SL == GS_TILE) return (row >> 4) * B + b;
  return scale_offset(row, b, B, SL == GS_MFMA);
}

template <int SL, bool SWI, int MT>
__global__ __launch_bounds__(1024) void gemv_kernel(GemvArgs a) {
  constexpr int R = SWI ? 2 : 1;
  extern __shared__ float red[];               // [waves][R][MT * 16 columns m][16 rows n]
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, nw = blockDim.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int grp = blockIdx.y;
  int64_t m_begin = 0, m_end = a.M;
  if (a.num_groups) {
    m_begin = a.offsets[grp];
    m_end = a.offsets[grp + 1];
    m_begin = m_begin < 0 ? 0 : m_begin;
    m_end = m_end > a.M ? a.M : m_end;
  }
  if (m_begin >= m_end) return;
  const int64_t n0 = (int64_t)blockIdx.x * 16, B = a.K >> 4;
  const uint8_t* wrow[R];
  const uint8_t* srow[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    int64_t row = n0 + c;
    row = (row < a.N ? row : a.N - 1) + r * a.N;
    wrow[r] = a.w + grp * a.w_group + row * a.ld_w;
    srow[r] = a.scales + grp * a.s_group + gemv_scale_offset<SL>(row, 0, B);
  }
  const float S = a.gs[grp];
  const int64_t chunks = (a.K + 127) >> 7;

  for (int64_t m0 = m_begin; m0 < m_end; m0 += 16 * MT) {
    const uint16_t* xrow[MT];
    bool have[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int64_t m = m0 + t * 16 + c;
      int64_t xr = m;
      have[t] = m < m_end;
      if (have[t] && a.row_index) xr = a.row_index[m];
      have[t] = have[t] && xr >= 0 && xr < a.x_rows;
      xrow[t] = a.x + (have[t] ? xr : 0) * a.ld_x;
    }
    f32x4 acc[R][MT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[r][t] = f32x4{0, 0, 0, 0};

#pragma unroll 2
    for (int64_t ch = wave; ch < chunks; ch += nw) {
      const int64_t k = ch * 128 + g * 32, b = k >> 4;
      // K % 16 == 0: a lane holds two blocks, one, or none
      const int nb = b + 1 < B ? 2 : b < B ? 1 : 0;
      uint4 w[R];
      uint32_t s[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        w[r] = make_uint4(0, 0, 0, 0);
        s[r] = 0;
        const int64_t so = SL == GS_MFMA ? (b >> 2) * 128 + (b & 3) : b;
        if (nb == 2) {
          __builtin_memcpy(&w[r], wrow[r] + (k >> 1), 16);
          uint16_t two;
          __builtin_memcpy(&two, srow[r] + so, 2);
          s[r] = two;
        } else if (nb == 1) {
          uint2 half;
          __builtin_memcpy(&half, wrow[r] + (k >> 1), 8);
          w[r].x = half.x;
          w[r].y = half.y;
          s[r] = srow[r][so];
        }
      }
      uint4 x[MT][4];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[t][j] = make_uint4(0, 0, 0, 0);
          if (have[t] && (j >> 1) < nb) x[t][j] = *reinterpret_cast<const uint4*>(xrow[t] + k + 8 * j);
        }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float s0 = e4m3_to_f32(s[r] & 0xFF), s1 = e4m3_to_f32(s[r] >> 8);
        const uint32_t ww[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8 av = e2m1x8_to_bf16(ww[j], j < 2 ? s0 : s1);
#pragma unroll
          for (int t = 0; t < MT; ++t)
            acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, __builtin_bit_cast(bf16x8, x[t][j]),
                                                                acc[r][t], 0, 0, 0);
        }
      }
    }
    // lane (c, g) holds column m = c, rows n = 4 g .. + 3 of each tile
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < MT; ++t)
        *reinterpret_cast<f32x4*>(&red[(((wave * R + r) * MT + t) * 16 + c) * 16 + 4 * g]) = acc[r][t];
    __syncthreads();
    const int64_t cols = m_end - m0 < 16 * MT ? m_end - m0 : 16 * MT;
    for (int i = threadIdx.x; i < (int)cols * 16; i += blockDim.x) {
      const int m = i >> 4, n = i & 15;
      float v[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        v[r] = 0.0f;
        for (int w = 0; w < nw; ++w) v[r] += red[((w * R + r) * MT * 16 + m) * 16 + n];
        v[r] *= S;
      }
      // SwiGLU on the binary32 sums: silu(g) u = g / (1 + exp(-g)) u
      const float out = SWI ? v[0] / (1.0f + expf(-v[0])) * v[R - 1] : v[0];
      if (n0 + n < a.N) a.y[(m0 + m) * a.ld_y + n0 + n] = (uint16_t)f32x2_to_bf16x2(out, 0.0f);
    }
    __syncthreads();
  }
}

template <int SL, bool SWI>
static hipError_t launch_gemv_sl(const GemvArgs& a, hipStream_t st) {
  // waves of a workgroup: about four K chunks each, 16 at most
  const int64_t chunks = (a.K + 127) >> 7;
  const int nw = chunks >= 64 ? 16 : chunks >= 32 ? 8 : chunks >= 8 ? 4 : chunks >= 2 ? 2 : 1;
  const int groups = a.num_groups ? a.num_groups : 1;
  const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)groups);
  const size_t lds = (size_t)nw * (SWI ? 2 : 1) * 256 * sizeof(float);
  hipLaunchKernelGGL((gemv_kernel<SL, SWI, 1>), grid, dim3(64 * nw), lds, st, a);
  return hipGetLastError();
}

hipError_t launch_nvfp4_gemv(const GemvArgs& a, GemvScales layout, bool swiglu, hipStream_t st) {
  switch (layout) {
    case GS_ROW: return swiglu ? launch_gemv_sl<GS_ROW, true>(a, st) : launch_gemv_sl<GS_ROW, false>(a, st);
    case GS_MFMA: return swiglu ? launch_gemv_sl<GS_MFMA, true>(a, st) : launch_gemv_sl<GS_MFMA, false>(a, st);
    default: return swiglu ? launch_gemv_sl<GS_TILE, true>(a, st) : launch_gemv_sl<GS_TILE, false>(a, st);
  }
}

}  // namespace mxq
