// Root-mean-square norm with the residual's addition and a quantized output,
// and its gradient.
//
//   h = bf16(x + r),  rstd = fl(1 / sqrt(mean(h^2) + eps)),  y = bf16(fl(fl(h rstd) w))
//
// h^2 of BF16 values is summed in binary64, in one order whatever the launch (a chunk's
// eight values in turn; then a tree over the chunks of equal index modulo 64;
// then a tree over those 64), so a row's outputs have the same bits whatever the
// number of rows and the kernel that the launcher picks for it: a sampler's
// single row equals the learner's.  BF16 y is quantized by the quantizers' own code,
// with the bytes that they give for y.
//
// Both kernels are bound by memory: a row is read once and stays in registers (a lane owns
// chunks of eight values, 16 bytes), every output leaves from there.  8192 rows of 4096
// with a residual, MXFP8 and its values: 303 MB in 55.8 us, 5.4 TB/s, where a large copy has
// 5.2; 32001 rows, NVFP4: 213 us; one row 2.6 us, of which a launch alone is about 2.
// What the backward reads much later (h, the codes' values) and dx go past the caches
// (that alone: MXFP8 62.4 -> 55.8 us, the gradient of 32768 rows 216.8 -> 200).

#include "lanes.h"
#include "layer_kernels.h"
#include "mxfp8_device.h"
#include "nvfp4_device.h"

namespace mxq {

namespace {

// (a[0] + a[1]) + (a[2] + a[3]) ..., N a power of two
template <int N>
__device__ __forceinline__ double tree_sum(const double* a) {
  if constexpr (N == 1) return a[0];
  else return tree_sum<N / 2>(a) + tree_sum<N / 2>(a + N / 2);
}

__device__ __forceinline__ double sum_squares8(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const double a = bf16_lo(w[i]), b = bf16_hi(w[i]);
    s = __builtin_fma(a, a, s);
    s = __builtin_fma(b, b, s);
  }
  return s;
}

__device__ __forceinline__ uint4 add8(uint4 a, uint4 b) {
  // a binary32 sum of two BF16 values that is inexact lies near the larger of
  // them, never near a border of BF16: the two roundings are one
  uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w}, o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = f32x2_to_bf16x2(bf16_lo(x[i]) + bf16_lo(y[i]), bf16_hi(x[i]) + bf16_hi(y[i]));
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ uint4 scaled8(uint4 h, float rstd, uint4 w) {
  uint32_t x[4] = {h.x, h.y, h.z, h.w}, g[4] = {w.x, w.y, w.z, w.w}, o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = f32x2_to_bf16x2((bf16_lo(x[i]) * rstd) * bf16_lo(g[i]), (bf16_hi(x[i]) * rstd) * bf16_hi(g[i]));
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// BF16 of eight E4M3 codes times a block scale: a power of two (s: its E8M0
// code; exact) or a binary32 value (s: its bits; one rounding, then BF16's).
template <bool F32S>
__device__ __forceinline__ uint4 fp8_values8(uint2 codes, uint32_t s) {
  const uint32_t w[2] = {codes.x, codes.y};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t word = w[i >> 1] >> (16 * (i & 1));
    const float a = e4m3_to_f32(word & 0xFF), b = e4m3_to_f32((word >> 8) & 0xFF);
    if constexpr (F32S) o[i] = f32x2_to_bf16x2(a * __uint_as_float(s), b * __uint_as_float(s));
    else o[i] = f32x2_to_bf16x2(__builtin_ldexpf(a, (int)s - 127), __builtin_ldexpf(b, (int)s - 127));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// LANES lanes (16 or 64) times WAVES waves hold a row, CH chunks a lane: chunk
// lane + LANES (wave CH + i).  16 lanes hold a short row of one chunk a lane, four rows a wave.
// A wave a row needs no barrier and wins with many rows (32768 of 1024 values, NVFP4:
// 55.7 us, 110.3 with four waves); more waves a row win with few (1100 of 4096, MXFP8: 10.9
// against 13.1) and with long ones, where two chunks a lane leave registers for four waves
// a SIMD (4096 rows of 16384, MXFP8: 109 us, 127 with eight chunks).
template <int LANES, int WAVES, int CH, int FMT>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void rmsnorm_kernel(NormArgs a) {
  static_assert(LANES == 64 || (LANES == 16 && WAVES == 1 && CH == 1), "rows of 16 lanes are short");
  constexpr int THREADS = WAVES == 1 ? 256 : 64 * WAVES;
  constexpr int ROWS = THREADS / (LANES * WAVES);            // of a workgroup
  constexpr bool FP8 = FMT == MXQ_FMT_MXFP8 || FMT == MXQ_FMT_FP8_B128 || FMT == MXQ_FMT_FP8_B128_F32;
  constexpr bool F32S = FMT == MXQ_FMT_FP8_B128_F32;
  constexpr int LPB = FMT == MXQ_FMT_MXFP8 ? 4 : 16;         // lanes of an FP8 block
  // two of each, used in turn: a wave still reading one is at most one barrier behind
  __shared__ double part_sum[2][WAVES > 1 ? WAVES : 1][WAVES > 1 ? 64 : 1];
  __shared__ uint32_t part_max[2][WAVES > 1 ? WAVES : 1];

  const int lane = threadIdx.x & (LANES - 1);
  const int wave = WAVES > 1 ? threadIdx.x >> 6 : 0;
  const int chunks = (int)(a.cols >> 3);
  int c[CH];
  uint4 w[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    c[i] = lane + LANES * (wave * CH + i);
    w[i] = c[i] < chunks ? load16(a.w + 8 * c[i]) : make_uint4(0, 0, 0, 0);
  }
  int turn = 0;
  // whole waves leave the loop together but where 16 lanes hold a row: there the
  // exchanges stay inside those lanes
  for (int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / (LANES * WAVES); row < a.rows;
       row += (int64_t)gridDim.x * ROWS, turn ^= 1) {
    uint4 h[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i)
      h[i] = c[i] < chunks ? load16(a.x + row * a.ld_x + 8 * c[i]) : make_uint4(0, 0, 0, 0);
    if (a.r) {
      uint4 r[CH];
#pragma unroll
      for (int i = 0; i < CH; ++i)
        r[i] = c[i] < chunks ? load16(a.r + row * a.ld_r + 8 * c[i]) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < CH; ++i) h[i] = add8(h[i], r[i]);
    }
    double s[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) s[i] = sum_squares8(h[i]);
    double sum = tree_sum<CH>(s);
    if constexpr (WAVES > 1) {
      part_sum[turn][wave][lane] = sum;
      __syncthreads();
      double p[WAVES];
#pragma unroll
      for (int i = 0; i < WAVES; ++i) p[i] = part_sum[turn][i][lane];
      sum = tree_sum<WAVES>(p);
    }
    sum = lanes_sum<LANES>(sum);
    const float rstd = (float)(1.0 / sqrt(sum / (double)a.cols + a.eps));
    if (a.rstd && lane == 0 && wave == 0) a.rstd[row] = rstd;
    if (a.h) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (c[i] < chunks) store16_once(a.h + row * a.ld_h + 8 * c[i], h[i]);
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) h[i] = scaled8(h[i], rstd, w[i]);        // y from here on
    if (a.y) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (c[i] < chunks) store16(a.y + row * a.ld_y + 8 * c[i], h[i]);
    }
    if constexpr (FP8) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        uint32_t m = absmax8(h[i]);
        m = umax(m, dpp_u32<0xB1>(m));
        m = umax(m, dpp_u32<0x4E>(m));
        if constexpr (LPB == 16) {
          m = umax(m, dpp_u32<0x141>(m));
          m = umax(m, dpp_u32<0x140>(m));
        }
        const uint32_t sc = blk_scale<F32S>(m);
        const uint2 code = blk_encode8<F32S>(h[i], sc);
        if (c[i] < chunks) {
          *reinterpret_cast<uint2*>(a.codes + row * a.ld_codes + 8 * c[i]) = code;
          if (c[i] % LPB == 0) blk_store<F32S>(a.scales, scale_offset(row, c[i] / LPB, chunks / LPB, a.mfma), sc);
          if (a.dq) store16_once(a.dq + row * a.ld_dq + 8 * c[i], fp8_values8<F32S>(code, sc));
        }
      }
    }
    if constexpr (FMT == MXQ_FMT_NVFP4) {
      uint32_t m[CH], top = 0;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        m[i] = amax8_bits(h[i]);
        m[i] = umax(m[i], dpp_u32<0xB1>(m[i]));
        top = umax(top, m[i]);
      }
      top = lanes_max<LANES>(top);
      if constexpr (WAVES > 1) {
        if (lane == 0) part_max[turn][wave] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WAVES; ++i) top = umax(top, part_max[turn][i]);
      }
      const float S = __uint_as_float(top) / 2688.0f;
      if (lane == 0 && wave == 0) a.gs[row] = S;
      const u32x4 none = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const BlockScale bs = nv_block_scale(__uint_as_float(m[i]), S);
        const uint32_t code =
            S < TINY_S ? nv_encode8<false, true>(h[i], bs.r, none) : nv_encode8<false, false>(h[i], bs.r, none);
        if (c[i] < chunks) {
          *reinterpret_cast<uint32_t*>(a.codes + row * a.ld_codes + 4 * c[i]) = code;
          if ((c[i] & 1) == 0) a.scales[scale_offset(row, c[i] >> 1, chunks >> 1, a.mfma)] = (uint8_t)bs.code;
          if (a.dq) store16_once(a.dq + row * a.ld_dq + 8 * c[i], nv_decode8(code, e4m3_to_f32(bs.code), S));
        }
      }
    }
  }
}

template <int LANES, int WAVES, int CH>
hipError_t launch_norm(const NormArgs& a, mxq_format fmt, hipStream_t st) {
  constexpr int THREADS = WAVES == 1 ? 256 : 64 * WAVES;
  constexpr int ROWS = THREADS / (LANES * WAVES);
  const int64_t need = (a.rows + ROWS - 1) / ROWS, most = 2048 * 256 / THREADS;
  const dim3 grid((unsigned)(need < most ? need : most)), block(THREADS);
  switch (fmt) {
    case MXQ_FMT_MXFP8:
      hipLaunchKernelGGL((rmsnorm_kernel<LANES, WAVES, CH, MXQ_FMT_MXFP8>), grid, block, 0, st, a);
      break;
    case MXQ_FMT_FP8_B128:
      hipLaunchKernelGGL((rmsnorm_kernel<LANES, WAVES, CH, MXQ_FMT_FP8_B128>), grid, block, 0, st, a);
      break;
    case MXQ_FMT_FP8_B128_F32:
      hipLaunchKernelGGL((rmsnorm_kernel<LANES, WAVES, CH, MXQ_FMT_FP8_B128_F32>), grid, block, 0, st, a);
      break;
    case MXQ_FMT_NVFP4:
      hipLaunchKernelGGL((rmsnorm_kernel<LANES, WAVES, CH, MXQ_FMT_NVFP4>), grid, block, 0, st, a);
      break;
    default:
      hipLaunchKernelGGL((rmsnorm_kernel<LANES, WAVES, CH, MXQ_FMT_BF16>), grid, block, 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, mxq_format fmt, hipStream_t st) {
  const int64_t n = a.cols;
  if (n <= 128) return launch_norm<16, 1, 1>(a, fmt, st);
  if (n <= 512) return launch_norm<64, 1, 1>(a, fmt, st);
  if (n <= 1024) return launch_norm<64, 1, 2>(a, fmt, st);
  // a wave a row where that makes two for every SIMD, else four and more
  if (a.rows >= 2048) {
    if (n <= 2048) return launch_norm<64, 1, 4>(a, fmt, st);
    if (n <= 4096) return launch_norm<64, 1, 8>(a, fmt, st);
  }
  if (n <= 4096) return launch_norm<64, 4, 2>(a, fmt, st);
  if (n <= 8192) return launch_norm<64, 8, 2>(a, fmt, st);
  if (n <= 16384) return launch_norm<64, 16, 2>(a, fmt, st);
  return launch_norm<64, 16, 4>(a, fmt, st);
}

// ------------------------------------------------------------------- gradient
//
//   g = dy w,  xhat = h rstd,  dx = rstd (g - xhat mean(g xhat)) + dres,  dw = sum over rows of dy xhat
//
// The row sum and dw are binary32.  TEAMS teams of WAVES waves hold a row each;
// a workgroup walks rows and keeps dw of its columns in registers; the teams'
// sums meet in LDS, the workgroup's go to the workspace, and a second kernel adds those,
// always in the same order (no atomics).  32768 rows of 4096 with dres: 1.07 GB in
// 186 us, 5.8 TB/s, 199.7 with one team a workgroup and 1024 workgroups; 1003 rows of 2048:
// 8.5 us, two launches (11.8 with a workgroup a row).

namespace {

// Keeps the compiler from holding what it computed of v before (binary32 values
// take twice the registers of v itself).
__device__ __forceinline__ void opaque(uint4& v) { asm volatile("" : "+v"(v.x), "+v"(v.y), "+v"(v.z), "+v"(v.w)); }

template <int WAVES, int TEAMS, int CH>
__global__ __launch_bounds__(64 * WAVES * TEAMS) void rmsnorm_backward_kernel(NormBwdArgs a) {
  constexpr int COLS = 512 * WAVES * CH;
  // the widest rows: 16 waves have 128 registers a lane, so the weight is read
  // where it is used, dres behind the row's sum, and nothing that was computed of
  // dy and h before is kept (4096 rows of 32768: 626 us with all of it in registers, 311 so)
  constexpr bool LEAN = COLS > 16384;
  __shared__ float part[2][TEAMS][WAVES];
  __shared__ float team_dw[TEAMS > 1 ? COLS : 1];
  const int lane = threadIdx.x & 63;
  const int wave = (threadIdx.x >> 6) % WAVES, team = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) / WAVES);
  const int chunks = (int)(a.cols >> 3);
  const float inv = 1.0f / (float)a.cols;
  int c[CH];
  uint4 w[CH];
  float dw[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    c[i] = lane + 64 * (wave * CH + i);
    if (!LEAN) w[i] = c[i] < chunks ? load16(a.w + 8 * c[i]) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  }
  int turn = 0;
  // every team takes every step, so that all waves meet at the barriers
  for (int64_t row0 = (int64_t)blockIdx.x * TEAMS; row0 < a.rows; row0 += (int64_t)gridDim.x * TEAMS, turn ^= 1) {
    const int64_t row = row0 + team;
    const bool live = TEAMS == 1 || row < a.rows;
    uint4 dy[CH], h[CH], r[CH];
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const bool has = live && c[i] < chunks;
      dy[i] = has ? load16(a.dy + row * a.ld_dy + 8 * c[i]) : zero;
      h[i] = has ? load16_once(a.h + row * a.ld_h + 8 * c[i]) : zero;
      if (!LEAN) r[i] = a.dres && has ? load16(a.dres + row * a.ld_dres + 8 * c[i]) : zero;
      if (LEAN) w[i] = has ? load16(a.w + 8 * c[i]) : zero;
    }
    const float rstd = live ? a.rstd[row] : 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const uint32_t y[4] = {dy[i].x, dy[i].y, dy[i].z, dy[i].w}, x[4] = {h[i].x, h[i].y, h[i].z, h[i].w};
      const uint32_t g[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float t0 = bf16_lo(y[j]) * (bf16_lo(x[j]) * rstd), t1 = bf16_hi(y[j]) * (bf16_hi(x[j]) * rstd);
        dw[i][2 * j] += t0;
        dw[i][2 * j + 1] += t1;
        s = __builtin_fmaf(t0, bf16_lo(g[j]), s);
        s = __builtin_fmaf(t1, bf16_hi(g[j]), s);
      }
    }
    s = lanes_sum<64>(s);
    if constexpr (WAVES > 1) {
      if (lane == 0) part[turn][team][wave] = s;
      __syncthreads();
      s = 0.0f;
#pragma unroll
      for (int i = 0; i < WAVES; ++i) s += part[turn][team][i];
    }
    const float m = s * inv;                                   // mean of g xhat
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (LEAN) {
        opaque(dy[i]);
        opaque(h[i]);
      }
      if (LEAN) {
        const bool has = live && c[i] < chunks;
        w[i] = has ? load16(a.w + 8 * c[i]) : zero;
        r[i] = a.dres && has ? load16(a.dres + row * a.ld_dres + 8 * c[i]) : zero;
      }
      const uint32_t y[4] = {dy[i].x, dy[i].y, dy[i].z, dy[i].w}, x[4] = {h[i].x, h[i].y, h[i].z, h[i].w};
      const uint32_t g[4] = {w[i].x, w[i].y, w[i].z, w[i].w}, d[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float t0 = __builtin_fmaf(-(bf16_lo(x[j]) * rstd), m, bf16_lo(y[j]) * bf16_lo(g[j]));
        const float t1 = __builtin_fmaf(-(bf16_hi(x[j]) * rstd), m, bf16_hi(y[j]) * bf16_hi(g[j]));
        o[j] = f32x2_to_bf16x2(__builtin_fmaf(rstd, t0, bf16_lo(d[j])), __builtin_fmaf(rstd, t1, bf16_hi(d[j])));
      }
      if (live && c[i] < chunks) store16_once(a.dx + row * a.ld_dx + 8 * c[i], make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
  if (!a.dw) return;                           // the same for all
  if constexpr (TEAMS > 1) {
    // the teams in turn, the last one keeps the sum
    for (int k = 0; k < TEAMS; ++k) {
      if (team == k) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          float4* p = reinterpret_cast<float4*>(team_dw + 8 * c[i]);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float4 t = k ? p[q] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            t = make_float4(t.x + dw[i][4 * q], t.y + dw[i][4 * q + 1], t.z + dw[i][4 * q + 2], t.w + dw[i][4 * q + 3]);
            dw[i][4 * q] = t.x;
            dw[i][4 * q + 1] = t.y;
            dw[i][4 * q + 2] = t.z;
            dw[i][4 * q + 3] = t.w;
            if (k < TEAMS - 1) p[q] = t;
          }
        }
      }
      __syncthreads();
    }
    if (team != TEAMS - 1) return;
  }
  float* p = a.part + (int64_t)blockIdx.x * a.cols;
#pragma unroll
  for (int i = 0; i < CH; ++i)
    if (c[i] < chunks) {
      float4* q = reinterpret_cast<float4*>(p + 8 * c[i]);
      q[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
      q[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
    }
}

// dw[c] = sum of the groups' part[g][c]: 32 columns a workgroup, eight lanes of
// four each; 128 lanes of groups, each its groups in turn, then in the order of the lanes.
__global__ __launch_bounds__(1024) void rmsnorm_dw_kernel(const float* part, int64_t groups, int64_t cols, float* dw) {
  __shared__ float4 s[128][9];
  const int x = threadIdx.x & 7, y = threadIdx.x >> 3;
  const int64_t c = ((int64_t)blockIdx.x * 8 + x) * 4;
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < cols) {
#pragma unroll 4
    for (int64_t g = y; g < groups; g += 128) {
      const float4 v = *reinterpret_cast<const float4*>(part + g * cols + c);
      sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
    }
  }
  s[y][x] = sum;
  __syncthreads();
  for (int n = 64; n >= 1; n /= 2) {
    if (y < n) {
      const float4 v = s[y + n][x];
      sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
      s[y][x] = sum;
    }
    __syncthreads();
  }
  if (y == 0 && c < cols) *reinterpret_cast<float4*>(dw + c) = sum;
}

// The kernel's shape for a number of columns, and the workgroups that it runs on.
struct BwdShape {
  int teams;
  int64_t most;
};
BwdShape bwd_shape(int64_t cols) {
  if (cols <= 512) return {4, 1024};
  if (cols <= 2048) return {4, 512};
  if (cols <= 4096) return {2, 512};
  return {1, cols <= 16384 ? 512 : 256};
}

template <int WAVES, int TEAMS, int CH>
void launch_bwd(const NormBwdArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)norm_bwd_groups(a.rows, a.cols)), block(64 * WAVES * TEAMS);
  hipLaunchKernelGGL((rmsnorm_backward_kernel<WAVES, TEAMS, CH>), grid, block, 0, st, a);
}

}  // namespace

int64_t norm_bwd_groups(int64_t rows, int64_t cols) {
  const BwdShape s = bwd_shape(cols);
  const int64_t need = (rows + s.teams - 1) / s.teams;
  return need < s.most ? need : s.most;
}

hipError_t launch_rmsnorm_backward(const NormBwdArgs& a, hipStream_t st) {
  const int64_t n = a.cols;
  if (a.rows == 0) {}                          // no rows: a sum of nothing
  else if (n <= 512) launch_bwd<1, 4, 1>(a, st);
  else if (n <= 2048) launch_bwd<2, 4, 2>(a, st);
  else if (n <= 4096) launch_bwd<4, 2, 2>(a, st);
  else if (n <= 8192) launch_bwd<8, 1, 2>(a, st);
  else if (n <= 16384) launch_bwd<16, 1, 2>(a, st);
  else launch_bwd<16, 1, 4>(a, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.dw) return e;
  hipLaunchKernelGGL(rmsnorm_dw_kernel, dim3((unsigned)((n + 31) / 32)), dim3(1024), 0, st, a.part,
                     norm_bwd_groups(a.rows, n), n, a.dw);
  return hipGetLastError();
}

}  // namespace mxq
