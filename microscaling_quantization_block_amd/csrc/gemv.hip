// Few BF16 rows times NVFP4 weights: y[m, n] = sum_k x[m, k] value(c) s_b S.
//
// The products are exact: an E2M1 code times its E4M3 block scale has at most
// six significant bits and lies in 2^-10 .. 2688, so it is a BF16 number, and
// the BF16 matrix instruction multiplies it with x unrounded and sums in
// binary32.  S leaves the sum and multiplies it once, in binary32; one
// rounding to BF16 ends the chain.
//
// Three kernels; all are bound by the weights' bytes (one row through 4096 x
// 14336: 33 MB in 10.2 us; 13 rows through 24576 x 4096: 57 MB in 20.9 us, 2.7
// TB/s, where a large copy has 4.8), the short ones by the latency of one load
// and of the join of the partial sums.
//
// This first one takes any shape and any number of rows.  A workgroup owns 16 RT
// weight rows (with SwiGLU as many gate rows and their up rows) and all of K;
// its waves take 256-wide K chunks in turn (a whole 128-byte line of codes per
// row) and their partial tiles meet in LDS, so there are many loads in flight
// for a matrix with few rows and no second launch.  The weights are the left
// operand: lane (c, g) = (lane % 16, lane / 16) reads 32 bytes, the codes k0 +
// 64 g .. + 63 of row c, with their four scales in one word, and feeds them to
// eight matrix instructions eight at a time; x is read in the same order, so k
// is permuted alike on both sides and nothing is shuffled.  (Lanes g next to
// each other along K, in 8-byte pieces, touch half as many lines per load but
// need more loads: 23.4 us against 20.7 for 8 rows through 4096 x 14336.)
// R > 1 because x comes through the caches: 16 rows of x are four times the
// bytes of 16 rows of codes.  A chunk's loads are in flight while the one
// before it is multiplied; no load in the loop depends on a branch (lanes
// without a row of x read some row, whose column is dropped at the end), so the
// waits count them.

#include "mxq_device.h"
#include "decode_kernels.h"
#include "mxq_kernels.h"

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

// R tiles of 16 weight rows (with SwiGLU tile 2 t holds gate rows and tile
// 2 t + 1 their up rows), MT tiles of 16 rows of x.
template <int SL, bool SWI, int R, int MT>
__global__ __launch_bounds__(R == 1 && MT == 1 ? 1024 : 512) void gemv_kernel(GemvArgs a) {
  constexpr int RT = SWI ? R / 2 : R;          // tiles of output columns
  extern __shared__ float red[];               // [waves][R][MT * 16 columns m][16 rows n]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), nw = blockDim.x >> 6;
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
  const int64_t n0 = (int64_t)blockIdx.x * 16 * RT, B = a.K >> 4;
  const int full = (int)(a.K >> 8), rest = (int)(a.K & 255);   // whole chunks, and what is left
  // the lane's codes and scales of chunk 0; a chunk adds 128 bytes and 16 (MFMA: 512) bytes of scales
  const uint8_t* wp[R];
  const uint8_t* sp[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    int64_t row = n0 + (SWI ? r >> 1 : r) * 16 + c;
    row = (row < a.N ? row : a.N - 1) + (SWI && (r & 1) ? a.N : 0);
    wp[r] = a.w + grp * a.w_group + row * a.ld_w + 32 * g;
    sp[r] = a.scales + grp * a.s_group + gemv_scale_offset<SL>(row, 0, B) + (SL == GS_MFMA ? 128 : 4) * g;
  }
  constexpr int S_CHUNK = SL == GS_MFMA ? 512 : 16;
  const float S = a.gs[grp];

  for (int64_t m0 = m_begin; m0 < m_end; m0 += 16 * MT) {
    const uint16_t* xp[MT];
    bool have[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int64_t m = m0 + t * 16 + c;
      int64_t xr = m;
      have[t] = m < m_end;
      if (have[t] && a.row_index) xr = a.row_index[m];
      have[t] = have[t] && xr >= 0 && xr < a.x_rows;
      xp[t] = a.x + (have[t] ? xr : 0) * a.ld_x + 64 * g;
    }
    f32x4 acc[R][MT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[r][t] = f32x4{0, 0, 0, 0};

    struct Chunk {
      uint4 w[R][2], x[MT][8];
      uint32_t s[R];
    };
    auto load = [&](Chunk& k, int ch) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        __builtin_memcpy(&k.w[r][0], wp[r] + (int64_t)ch * 128, 16);
        __builtin_memcpy(&k.w[r][1], wp[r] + (int64_t)ch * 128 + 16, 16);
        __builtin_memcpy(&k.s[r], sp[r] + (int64_t)ch * S_CHUNK, 4);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) k.x[t][j] = *reinterpret_cast<const uint4*>(xp[t] + (int64_t)ch * 256 + 8 * j);
    };
    auto multiply = [&](const Chunk& k) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t ww[8] = {k.w[r][0].x, k.w[r][0].y, k.w[r][0].z, k.w[r][0].w,
                                k.w[r][1].x, k.w[r][1].y, k.w[r][1].z, k.w[r][1].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bf16x8 av = e2m1x8_to_bf16(ww[j], e4m3_to_f32((k.s[r] >> (8 * (j >> 1))) & 0xFF));
#pragma unroll
          for (int t = 0; t < MT; ++t)
            acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, __builtin_bit_cast(bf16x8, k.x[t][j]), acc[r][t],
                                                                0, 0, 0);
        }
      }
    };

    // the wave's whole chunks: wave, wave + nw, ...
    if (full > wave) {
      Chunk k[2];
      const int last = wave + (full - wave - 1) / nw * nw;
      load(k[0], wave);
      int ch = wave;
      while (true) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          load(k[1 - h], min(ch + nw, last));  // behind the last one: that again
          multiply(k[h]);
          ch += nw;
          if (ch > last) goto done;
        }
      }
    }
  done:
    // what is left of K: a lane holds up to four blocks
    if (rest && wave == full % nw) {
      const int nb = min(max((rest >> 4) - 4 * g, 0), 4);
      Chunk k;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint8_t* w = wp[r] + (int64_t)full * 128;
        const uint8_t* s = sp[r] + (int64_t)full * S_CHUNK;
        k.s[r] = 0;
        uint2 d[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          d[b] = make_uint2(0, 0);
          if (b < nb) {
            __builtin_memcpy(&d[b], w + 8 * b, 8);
            k.s[r] |= (uint32_t)s[b] << (8 * b);
          }
        }
        k.w[r][0] = make_uint4(d[0].x, d[0].y, d[1].x, d[1].y);
        k.w[r][1] = make_uint4(d[2].x, d[2].y, d[3].x, d[3].y);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          k.x[t][j] = make_uint4(0, 0, 0, 0);
          if ((j >> 1) < nb) k.x[t][j] = *reinterpret_cast<const uint4*>(xp[t] + (int64_t)full * 256 + 8 * j);
        }
      multiply(k);
    }
    // lane (c, g) holds column m = c, rows n = 4 g .. + 3 of each tile
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < MT; ++t)
        *reinterpret_cast<f32x4*>(&red[(((wave * R + r) * MT + t) * 16 + c) * 16 + 4 * g]) =
            have[t] ? acc[r][t] : f32x4{0, 0, 0, 0};
    __syncthreads();
    const int cols = (int)(m_end - m0 < 16 * MT ? m_end - m0 : 16 * MT);
    for (int i = threadIdx.x; i < cols * 16 * RT; i += blockDim.x) {
      const int n = i & 15, rt = (i >> 4) % RT, m = i / (16 * RT);
      float v[2];
#pragma unroll
      for (int e = 0; e < (SWI ? 2 : 1); ++e) {
        const int r = SWI ? 2 * rt + e : rt;
        v[e] = 0.0f;
        for (int w = 0; w < nw; ++w) v[e] += red[((w * R + r) * MT * 16 + m) * 16 + n];
        v[e] *= S;
      }
      // SwiGLU on the binary32 sums: silu(g) u = g / (1 + exp(-g)) u
      const float out = SWI ? v[0] / (1.0f + expf(-v[0])) * v[1] : v[0];
      const int64_t col = n0 + rt * 16 + n;
      if (col < a.N) a.y[(m0 + m) * a.ld_y + col] = (uint16_t)f32x2_to_bf16x2(out, 0.0f);
    }
    __syncthreads();
  }
}

template <int SL, bool SWI, int R, int MT>
static hipError_t launch_gemv_as(const GemvArgs& a, hipStream_t st) {
  constexpr int RT = SWI ? R / 2 : R;
  // a wave per chunk, as far as there is room
  const int chunks = (int)((a.K + 255) >> 8), most = R == 1 && MT == 1 ? 16 : 8, per = (chunks + most - 1) / most;
  const int nw = (chunks + per - 1) / per;
  const dim3 grid((unsigned)((a.N + 16 * RT - 1) / (16 * RT)), (unsigned)(a.num_groups ? a.num_groups : 1));
  const size_t lds = (size_t)nw * R * MT * 256 * sizeof(float);
  hipLaunchKernelGGL((gemv_kernel<SL, SWI, R, MT>), grid, dim3(64 * nw), lds, st, a);
  return hipGetLastError();
}

// ------------------------------------------------------------------ a few rows
//
// For one or two rows of x per matrix the matrix instruction has little to do,
// and its operand layout reads 16 rows at once, 16 bytes each, which
// the memory path takes apart.  Here the lanes lie along K: a lane holds 32
// codes of a row, 16 bytes, and a load of a wave is one kilobyte of one row
// (or of 64 / LPR rows where K is short).  A wave reads 16 such pieces of
// neighbouring rows, all in flight at once, and multiplies them with its part
// of x, which stays in registers: codes to BF16 pairs (exact), v_dot2 in
// binary32, the two blocks' sums times their E4M3 scales, then a sum over the
// lanes: over the 16 of a group piece by piece, after which lane c keeps piece
// c, and over the groups for all 16 pieces at once.  Waves take different
// rows, and where K is longer than 32 LPR different parts of K, which meet in
// LDS.

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int DOT_ITEMS = 16;

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
// Sum over the 16 lanes of a group, in every one of them.
__device__ __forceinline__ float sum16(float v) {
  v = dpp_add<0xB1>(v);                        // quads: neighbours, pairs
  v = dpp_add<0x4E>(v);
  v = dpp_add<0x141>(v);                       // mirrors: halves of 16, 16
  return dpp_add<0x140>(v);
}
// Sum over the lane groups of a row (LPR / 16 of them).
template <int LPR>
__device__ __forceinline__ float sum_groups(float v) {
  if (LPR >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  if (LPR >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  return v;
}

// Eight codes times eight values of x (as BF16 pairs).
__device__ __forceinline__ float dot8(uint32_t w, uint4 x, float acc) {
  const bf16x2 c[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1),
                       __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3)};
  const uint32_t xx[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    acc = __builtin_amdgcn_fdot2_f32_bf16(c[i], __builtin_bit_cast(bf16x2, xx[i]), acc, false);
  return acc;
}

// MM rows of x at a time (one where no matrix has more on average: two need 32
// more registers); ks waves of a workgroup share a row's K.
template <int SL, bool SWI, int LPR, int MM>
__global__ __launch_bounds__(512, MM == 1 ? 4 : 3) void gemv_dot_kernel(GemvArgs a, int ks) {
  constexpr int ITEMS = DOT_ITEMS, RPL = 64 / LPR;             // rows of a load
  constexpr int ROWS = ITEMS * RPL, OUT = SWI ? ROWS / 2 : ROWS;   // of a wave: weight rows, output columns
  constexpr int RUN = SWI ? ITEMS / 2 : ITEMS;                 // neighbouring rows of a lane
  __shared__ float part[8][ROWS * MM];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kpart = wave % ks, rpart = wave / ks, rs = (int)(blockDim.x >> 6) / ks;
  const int grp = blockIdx.y;
  int64_t m_begin = 0, m_end = a.M;
  if (a.num_groups) {
    m_begin = a.offsets[grp];
    m_end = a.offsets[grp + 1];
    m_begin = m_begin < 0 ? 0 : m_begin;
    m_end = m_end > a.M ? a.M : m_end;
  }
  if (m_begin >= m_end) return;
  const int64_t B = a.K >> 4;
  const int64_t n0 = ((int64_t)blockIdx.x * rs + rpart) * OUT;   // first output column of the wave
  // the lane's codes: k0 .. k0 + 31, of which those from `from` on count (the
  // last piece of a K that is no multiple of 32 overlaps the one before)
  const int64_t from = ((int64_t)kpart * LPR + lane % LPR) * 32;
  const int64_t k0 = from + 32 <= a.K ? from : a.K - 32, b0 = k0 >> 4;
  uint4 w[ITEMS];
  uint32_t s[ITEMS];                           // the lane's two scales, in the low half
  const uint8_t* scales = a.scales + grp * a.s_group;
#pragma unroll
  for (int r = 0; r < ITEMS / RUN; ++r) {      // SwiGLU: gate rows, then up rows
    // rows behind the last one are read as rows before it, and not written
    const int64_t first = n0 + (int64_t)(lane / LPR) * RUN;
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      const int64_t row = (first + i < a.N ? first + i : a.N - 1) + r * a.N;
      __builtin_memcpy(&w[r * RUN + i], a.w + grp * a.w_group + row * a.ld_w + (k0 >> 1), 16);
      if (SL == GS_ROW) {
        uint16_t two;
        __builtin_memcpy(&two, scales + row * B + b0, 2);
        s[r * RUN + i] = two;
      }
    }
    if (SL == GS_TILE) {                       // one tile row: N and the first row are multiples of RUN
      uint16_t two;
      __builtin_memcpy(&two, scales + (((first < a.N ? first : 0) + r * a.N) >> 4) * B + b0, 2);
#pragma unroll
      for (int i = 0; i < RUN; ++i) s[r * RUN + i] = two;
    }
    if (SL == GS_MFMA) {                       // four rows' words of four blocks are neighbours
      const int64_t row = (first < a.N ? first : 0) + r * a.N;
      const uint8_t* p = scales + ((row >> 5) * (B >> 2) + (b0 >> 2)) * 128 + (row & 31) * 4;
#pragma unroll
      for (int i = 0; i < RUN; i += 4) {
        uint32_t word[4];                      // scales may lie at any address
        __builtin_memcpy(word, p + 4 * i, 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[r * RUN + i + j] = word[j] >> (8 * (b0 & 3));
      }
    }
  }
  const float S = a.gs[grp];
  for (int64_t m0 = m_begin; m0 < m_end; m0 += MM) {
    uint4 x[MM][4];
#pragma unroll
    for (int m = 0; m < MM; ++m) {
      int64_t xr = m0 + m;
      bool have = xr < m_end;
      if (have && a.row_index) xr = a.row_index[xr];
      have = have && xr >= 0 && xr < a.x_rows;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[m][j] = make_uint4(0, 0, 0, 0);
        const int64_t k = k0 + 8 * j;
        if (have && k >= from && from < a.K) x[m][j] = *reinterpret_cast<const uint4*>(a.x + xr * a.ld_x + k);
      }
    }
    float sums[MM] = {};
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      // (keeps the conversions inside the loop over m0: outside they would take
      // four times the registers)
      asm("" : "+v"(w[i].x), "+v"(w[i].y), "+v"(w[i].z), "+v"(w[i].w), "+v"(s[i]));
      const float s0 = e4m3_to_f32(s[i] & 0xFF), s1 = e4m3_to_f32((s[i] >> 8) & 0xFF);
#pragma unroll
      for (int m = 0; m < MM; ++m) {
        const float d0 = dot8(w[i].y, x[m][1], dot8(w[i].x, x[m][0], 0.0f));
        const float d1 = dot8(w[i].w, x[m][3], dot8(w[i].z, x[m][2], 0.0f));
        const float v = sum16(__builtin_fmaf(d0, s0, d1 * s1));
        sums[m] = (lane & 15) == i ? v : sums[m];
      }
    }
    // lane c of a row's first group: weight row RUN (lane / LPR) + c % RUN of the gate or up rows
#pragma unroll
    for (int m = 0; m < MM; ++m) {
      sums[m] = sum_groups<LPR>(sums[m]);
      const int i = lane & 15;
      if (lane % LPR < 16) part[wave][(i / RUN * OUT + lane / LPR * RUN + i % RUN) * MM + m] = sums[m];
    }
    __syncthreads();
    const int cols = (int)(m_end - m0 < MM ? m_end - m0 : MM);
    for (int t = threadIdx.x; t < rs * OUT * cols; t += blockDim.x) {
      const int n = t % OUT, r = t / OUT % rs, m = t / (OUT * rs);
      float v[2] = {0.0f, 0.0f};
#pragma unroll
      for (int e = 0; e < (SWI ? 2 : 1); ++e) {
        for (int k = 0; k < ks; ++k) v[e] += part[r * ks + k][(n + e * OUT) * MM + m];
        v[e] *= S;
      }
      const float out = SWI ? v[0] / (1.0f + expf(-v[0])) * v[1] : v[0];
      const int64_t col = ((int64_t)blockIdx.x * rs + r) * OUT + n;
      if (col < a.N) a.y[(m0 + m) * a.ld_y + col] = (uint16_t)f32x2_to_bf16x2(out, 0.0f);
    }
    __syncthreads();
  }
}

template <int SL, bool SWI, int LPR, int MM>
static hipError_t launch_dot_as(const GemvArgs& a, hipStream_t st) {
  const int ks = (int)((a.K + 32 * LPR - 1) / (32 * LPR)), rs = ks > 4 ? 1 : 4 / ks;
  const int64_t out = (int64_t)rs * DOT_ITEMS * (64 / LPR) / (SWI ? 2 : 1);
  const dim3 grid((unsigned)((a.N + out - 1) / out), (unsigned)(a.num_groups ? a.num_groups : 1));
  hipLaunchKernelGGL((gemv_dot_kernel<SL, SWI, LPR, MM>), grid, dim3(64 * ks * rs), 0, st, a, ks);
  return hipGetLastError();
}

template <int SL, bool SWI>
static hipError_t launch_dot_sl(const GemvArgs& a, bool one, hipStream_t st) {
  if (a.K <= 512) return one ? launch_dot_as<SL, SWI, 16, 1>(a, st) : launch_dot_as<SL, SWI, 16, 2>(a, st);
  if (a.K <= 1024) return one ? launch_dot_as<SL, SWI, 32, 1>(a, st) : launch_dot_as<SL, SWI, 32, 2>(a, st);
  return one ? launch_dot_as<SL, SWI, 64, 1>(a, st) : launch_dot_as<SL, SWI, 64, 2>(a, st);
}

// ------------------------------------------------------------ x held in registers
//
// The matrix instruction again, for K up to 4096: a wave keeps its one or two
// chunks of x in registers (read once) and streams weight tiles past them, so
// only the weights move.  They come by loads that write LDS themselves, whole
// 128-byte lines of eight lanes each, AHEAD items in advance; no register
// waits for them and no barrier is needed, since a wave reads only what it
// loaded.  In LDS the 16-byte pieces of row c are exchanged by c / 2, so that
// the 16 rows' pieces that the operand layout reads together lie in different
// banks.  After each tile the waves' partial sums meet in LDS (two buffers, one
// barrier per tile).

constexpr int ITEM = 2048 + 256;               // LDS bytes: 16 rows of 256 codes, 16 rows of 16 scales

__device__ __forceinline__ void gemv_load16(const void* p, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void gemv_load4(const void* p, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(p), "{m0}"(lds) : "memory");
}

// AHEAD: items in flight behind the one being multiplied.  Three for eight
// waves (13 rows through 24576 x 4096: 21.1 us, four 21.5, two 25.9); two where
// a few waves are enough for K, for more workgroups on a compute unit (64 tokens
// through 128 experts, 2048 x 768: 32.5 us, three 35.6, four 37.7).
template <int SL, bool SWI, int XC, int AHEAD>
__global__ __launch_bounds__(512, 2) void gemv_stream_kernel(GemvArgs a, int tiles_per_wg) {
  constexpr int R = SWI ? 2 : 1, PER = R * XC; // items of a tile: weight tiles times chunks
  extern __shared__ __attribute__((aligned(16))) uint8_t s_gemv[];   // [waves][AHEAD + 1] items, then the partial sums
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), nw = blockDim.x >> 6;
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
  const int64_t B = a.K >> 4;
  const int tiles = (int)((a.N + 15) >> 4), t0 = blockIdx.x * tiles_per_wg, t1 = min(t0 + tiles_per_wg, tiles);
  if (t0 >= t1) return;
  const int chunks = (int)((a.K + 255) >> 8);
  const float S = a.gs[grp];
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(s_gemv) + wave * (AHEAD + 1) * ITEM;
  const uint8_t* ring = s_gemv + wave * (AHEAD + 1) * ITEM;
  float* red = reinterpret_cast<float*>(s_gemv + nw * (AHEAD + 1) * ITEM);   // [2][waves][R][16 m][16 n]

  // what a lane loads of an item: of rows lane / 8 and 8 + lane / 8 the 16-byte piece that belongs at
  // place lane % 8, and of row lane / 4 the four scales lane % 4
  const uint8_t* wbase = a.w + grp * a.w_group;
  const uint8_t* sbase = a.scales + grp * a.s_group;
  auto issue = [&](int item, int slot) {       // item = (tile - t0) * PER + r * XC + x; behind the last: some item again
    const int tile = min(t0 + item / PER, t1 - 1), r = item % PER / XC, x = item % XC;
    const int ch = min(wave + x * nw, chunks - 1);
    const int64_t k0 = (int64_t)ch * 256;
    const int left = (int)(a.K - k0 < 256 ? a.K - k0 : 256);   // a multiple of 64
    const uint32_t lds = lds0 + slot * ITEM;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");         // the slot's last readers have their values
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int lr = 8 * h + (lane >> 3);
      int piece = (lane & 7) ^ (lr >> 1);
      piece = 32 * piece < left ? piece : 0;   // behind K: any codes, x is zero there
      int64_t row = (int64_t)tile * 16 + lr;
      row = (row < a.N ? row : a.N - 1) + (SWI && r ? a.N : 0);
      gemv_load16(wbase + row * a.ld_w + (k0 >> 1) + 16 * piece, lds + 1024 * h);
    }
    const int word = 64 * (lane & 3) < left ? lane & 3 : 0;
    int64_t row = (int64_t)tile * 16 + (lane >> 2);
    row = (row < a.N ? row : a.N - 1) + (SWI && r ? a.N : 0);
    gemv_load4(sbase + gemv_scale_offset<SL>(row, (k0 >> 4) + 4 * word, B), lds + 2048);
  };

  for (int64_t m0 = m_begin; m0 < m_end; m0 += 16) {
    // x: lane (c, g) holds row m0 + c, the values 64 g + 8 j of its chunks; zero where there is none
    uint4 x[XC][8];
    {
      const int64_t m = m0 + c;
      int64_t xr = m;
      bool have = m < m_end;
      if (have && a.row_index) xr = a.row_index[m];
      have = have && xr >= 0 && xr < a.x_rows;
#pragma unroll
      for (int q = 0; q < XC; ++q) {
        const int64_t k = (int64_t)(wave + q * nw) * 256 + 64 * g;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[q][j] = make_uint4(0, 0, 0, 0);
        if (have && k < a.K)
#pragma unroll
          for (int j = 0; j < 8; ++j) x[q][j] = *reinterpret_cast<const uint4*>(a.x + xr * a.ld_x + k + 8 * j);
      }
    }
    const int cols = (int)(m_end - m0 < 16 ? m_end - m0 : 16);
    // nothing of the compiler's is in flight from here on but stores of y, which a wait may take for loads
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    for (int i = 0; i < AHEAD; ++i) issue(i, i);
    int item = 0, slot = 0;
    for (int t = t0; t < t1; ++t) {
      f32x4 acc[R];
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        const int r = q / XC, xi = q % XC;
        issue(item + AHEAD, slot ? slot - 1 : AHEAD);
        asm volatile("s_waitcnt vmcnt(%0)" ::"i"(3 * AHEAD) : "memory");
        const uint8_t* it = ring + slot * ITEM;
        const uint4 w0 = *reinterpret_cast<const uint4*>(it + c * 128 + (((2 * g) ^ (c >> 1)) << 4));
        const uint4 w1 = *reinterpret_cast<const uint4*>(it + c * 128 + (((2 * g + 1) ^ (c >> 1)) << 4));
        const uint32_t s = *reinterpret_cast<const uint32_t*>(it + 2048 + 16 * c + 4 * g);
        const uint32_t ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bf16x8 av = e2m1x8_to_bf16(ww[j], e4m3_to_f32((s >> (8 * (j >> 1))) & 0xFF));
          acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, __builtin_bit_cast(bf16x8, x[xi][j]), acc[r], 0, 0, 0);
        }
        ++item;
        slot = slot == AHEAD ? 0 : slot + 1;
      }
      float* buf = red + (t & 1) * nw * R * 256;
#pragma unroll
      for (int r = 0; r < R; ++r) *reinterpret_cast<f32x4*>(&buf[((wave * R + r) * 16 + c) * 16 + 4 * g]) = acc[r];
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      for (int i = threadIdx.x; i < cols * 16; i += blockDim.x) {
        const int n = i & 15, m = i >> 4;
        float v[2];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          v[r] = 0.0f;
          for (int w = 0; w < nw; ++w) v[r] += buf[((w * R + r) * 16 + m) * 16 + n];
          v[r] *= S;
        }
        const float out = SWI ? v[0] / (1.0f + expf(-v[0])) * v[R - 1] : v[0];
        const int64_t col = (int64_t)t * 16 + n;
        if (col < a.N) a.y[(m0 + m) * a.ld_y + col] = (uint16_t)f32x2_to_bf16x2(out, 0.0f);
      }
    }
    // the loads behind the last item must not write LDS after this
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }
}

template <int SL, bool SWI, int XC, int AHEAD>
static hipError_t launch_stream_as(const GemvArgs& a, int nw, hipStream_t st) {
  const int lds = nw * (AHEAD + 1) * ITEM + 2 * nw * (SWI ? 2 : 1) * 1024;
  static std::atomic<uint32_t> done{0};
  hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(&gemv_stream_kernel<SL, SWI, XC, AHEAD>), 160 * 1024, done);
  if (e != hipSuccess) return e;
  const int64_t groups = a.num_groups ? a.num_groups : 1, tiles = (a.N + 15) / 16;
  // as many workgroups as the chip holds at once, twice that for groups, of which some are empty
  const int64_t resident = 256 * (160 * 1024 / lds), want = a.num_groups ? 2 * resident : resident;
  const int64_t wgs = want / groups < 1 ? 1 : want / groups > tiles ? tiles : want / groups;
  const int64_t per = (tiles + wgs - 1) / wgs;
  const dim3 grid((unsigned)((tiles + per - 1) / per), (unsigned)groups);
  hipLaunchKernelGGL((gemv_stream_kernel<SL, SWI, XC, AHEAD>), grid, dim3(64 * nw), lds, st, a, (int)per);
  return hipGetLastError();
}

// Whole words and pieces: what its loads need.
static bool can_stream(const GemvArgs& a) {
  return a.K % 64 == 0 && a.K <= 4096 && a.ld_w % 16 == 0 && (reinterpret_cast<uintptr_t>(a.scales) & 3) == 0;
}

// Which kernel, by the rows per matrix on average and by the 16-row weight tiles
// of all matrices.  Measured, weights from memory:
//   lanes along K up to two rows: 2 rows through 4096 x 14336 12.9 us, tiles 16.6;
//     3 rows through 24576 x 4096 23.4 us, streamed 18.4.
//   streamed up to 16 rows: 8 rows through 4096 x 4096 8.3 us; lanes along K
//     16.8.  With more rows the weights come again for each 16 of them, from a
//     cache, which pays where x is long and there are many tiles: 32 rows
//     through 24576 x 4096 37.7 us, tiles 50.0; but 32 rows through 4096 x 4096
//     16.3 and 16.1, 64 through sixteen 2048 x 768 24.4 and 16.9.
//   tiles for the rest: R tiles of a workgroup share its x, as few as let all
//     workgroups run at once.  8 rows, R = 1, 2, 4: 4096 x 14336 20.7, 22.0,
//     33.4 us; 8192 x 8192 31, 17.3, 31; 16384 x 5120 36.1, 21.8, 19.1.
template <int SL, bool SWI>
static hipError_t launch_gemv_sl(const GemvArgs& a, hipStream_t st) {
  const int64_t groups = a.num_groups ? a.num_groups : 1;
  const int64_t rows = (a.M + groups - 1) / groups;
  const int64_t tiles = (a.N + 15) / 16 * (SWI ? 2 : 1) * groups;
  if (rows <= 2 && a.K >= 32 && a.K <= 16384) return launch_dot_sl<SL, SWI>(a, rows == 1, st);
  if (can_stream(a) && (rows <= 16 || (tiles > 512 && a.K > 2048))) {
    const int chunks = (int)((a.K + 255) >> 8);
    if (chunks > 8) return launch_stream_as<SL, SWI, 2, 3>(a, (chunks + 1) / 2, st);
    return chunks > 4 ? launch_stream_as<SL, SWI, 1, 3>(a, chunks, st) : launch_stream_as<SL, SWI, 1, 2>(a, chunks, st);
  }
  const int R = tiles <= 256 ? 1 : tiles <= 512 ? 2 : 4;
  if (rows > 16) {
    if constexpr (!SWI)
      if (R == 1) return launch_gemv_as<SL, SWI, 1, 2>(a, st);
    return R == 4 ? launch_gemv_as<SL, SWI, 4, 2>(a, st) : launch_gemv_as<SL, SWI, 2, 2>(a, st);
  }
  if constexpr (!SWI)
    if (R == 1) return launch_gemv_as<SL, SWI, 1, 1>(a, st);
  return R == 4 ? launch_gemv_as<SL, SWI, 4, 1>(a, st) : launch_gemv_as<SL, SWI, 2, 1>(a, st);
}

hipError_t launch_nvfp4_gemv(const GemvArgs& a, GemvScales layout, bool swiglu, hipStream_t st) {
  switch (layout) {
    case GS_ROW: return swiglu ? launch_gemv_sl<GS_ROW, true>(a, st) : launch_gemv_sl<GS_ROW, false>(a, st);
    case GS_MFMA: return swiglu ? launch_gemv_sl<GS_MFMA, true>(a, st) : launch_gemv_sl<GS_MFMA, false>(a, st);
    default: return swiglu ? launch_gemv_sl<GS_TILE, true>(a, st) : launch_gemv_sl<GS_TILE, false>(a, st);
  }
}

}  // namespace mxq
