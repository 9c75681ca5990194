// Attention over an NVFP4 cache.
//
// For a query column (one token, one head): x_t = scale q . k_t over the
// context, o = sum_t softmax(x)_t v_t, with k_t = value(c) s_b S_t.  Computed in
// one pass over the cache with the running maximum m and sum l of the softmax.
//
// The products run on the 16x16x32 FP16 matrix instruction.  value(c) s_b is
// an FP16 number (at most six significant bits, 2^-10 .. 2688), so K and V
// enter exactly; a query row is scaled by a power of two to have its largest
// element in [2^13, 2^14), which keeps its eight significant bits down to 2^-27
// of that element.  S of K multiplies the logit.  S of V multiplies the
// weight: w_t = p_t S_t / Sref 2^15 with Sref a running power of two above
// every S_t seen, rounded to FP16 (11 bits, 29 binades before it turns
// subnormal).  Sums, maxima and logits are binary32.
//
// Orientation: logits are computed transposed, X^T = K Q^T (A = 16 tokens, B = 16
// query columns), and the output too, O^T = V^T W^T.  A lane then holds one
// column (lane % 16) in both, so the softmax statistics and every rescaling
// are lane-local but for one exchange over the four lane groups, and the
// weights W leave the first product in the register layout the second one
// reads: the order of the 32 contracted tokens is permuted alike on both
// sides.  Lane (c, g) reads D / 8 contiguous code bytes of token c for K (the
// D / 4 values from g D / 4 on; q is read in that order), and for V D / 32
// bytes of each of the tokens 4 g .. 4 g + 3 of both 16-token halves; a pair of
// tokens' nibbles is interleaved so that one conversion gives two
// neighbouring contraction elements.

#include "cache_device.h"

namespace mxq {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int ATT_WAVES = 4;
constexpr int TILE = 32;                       // tokens of one step of a wave
constexpr float NEG_INF = -__builtin_inff();

template <int SEL>
__device__ __forceinline__ f16x2 fp4_pair(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, SEL);
}
__device__ __forceinline__ f16x2 fp4_pair_at(uint32_t w, int sel) {
  return sel == 0 ? fp4_pair<0>(w) : sel == 1 ? fp4_pair<1>(w) : sel == 2 ? fp4_pair<2>(w) : fp4_pair<3>(w);
}
// E4M3 bytes 0, 1 (hi false) or 2, 3 as FP16 (exact).
template <bool HI>
__device__ __forceinline__ f16x2 e4m3_pair(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI);
}

// What a wave reads of one 32-token tile.
template <int D>
struct RawTile {
  uint32_t k[2][D / 32];        // [half][dword]: token c of the half, values g D / 4 + 8 j ..
  uint32_t ks[2];               // its D / 64 block scales
  uint32_t v[2][4][(D + 127) / 128];   // [half][token 4 g + i]
  uint32_t vs[2];               // block scales of those four tokens
  f32x4 kg[2], vg[2];           // second scales of those four tokens
  int64_t t0;                   // first token
  uint32_t valid;               // bit 4 half + i: token usable
};

template <int BYTES>
__device__ __forceinline__ uint32_t load_small(const uint8_t* p) {
  if (BYTES == 1) return *p;
  if (BYTES == 2) return *reinterpret_cast<const uint16_t*>(p);
  return *reinterpret_cast<const uint32_t*>(p);
}

template <int D>
__device__ __forceinline__ void load_tile(const CacheArgs& cc, int64_t b, int h, int64_t t0, int64_t t_begin,
                                          int64_t t_end, int c, int g, RawTile<D>& r) {
  constexpr int VB = D / 32;                   // V bytes of a lane and token
  const int P = 1 << cc.P_log2;
  r.t0 = t0;
  r.valid = 0;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int64_t t = t0 + 16 * s;
    int64_t page = page_of(cc, b, t);          // 16 tokens lie in one page
    const bool ok = page >= 0;
    page = ok ? page : 0;
    const int64_t row = (int64_t)h * P + (t & (P - 1));
    const uint8_t* kc = cc.kc + page * cc.pc + (row + c) * (D / 2) + g * (D / 8);
    if (D == 64) {
      const uint2 w = *reinterpret_cast<const uint2*>(kc);
      r.k[s][0] = w.x, r.k[s][1] = w.y;
    } else {
#pragma unroll
      for (int j = 0; j < D / 128; ++j) {
        const uint4 w = *reinterpret_cast<const uint4*>(kc + 16 * j);
        r.k[s][4 * j] = w.x, r.k[s][4 * j + 1] = w.y, r.k[s][4 * j + 2] = w.z, r.k[s][4 * j + 3] = w.w;
      }
    }
    r.ks[s] = load_small<D / 64>(cc.ks + page * cc.psc + (row + c) * (D / 16) + g * (D / 64));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* vc = cc.vc + page * cc.pc + (row + 4 * g + i) * (D / 2) + c * VB;
      if (VB == 8) {
        const uint2 w = *reinterpret_cast<const uint2*>(vc);
        r.v[s][i][0] = w.x, r.v[s][i][(D + 127) / 128 - 1] = w.y;
      } else {
        r.v[s][i][0] = load_small<VB == 2 ? 2 : 4>(vc);
      }
    }
    const int vblk = c * (D / 16) / 16;
    uint32_t vs = *reinterpret_cast<const uint32_t*>(
        cc.vs + page * cc.psc + ((int64_t)h * (D / 16) + vblk) * P + (t & (P - 1)) + 4 * g);
    r.kg[s] = *reinterpret_cast<const f32x4*>(cc.kg + page * cc.pg + row + 4 * g);
    f32x4 vg = *reinterpret_cast<const f32x4*>(cc.vg + page * cc.pg + row + 4 * g);
    // a token outside the range, or without a page, may hold any bytes: its
    // V scales become zero here and its logit -inf later
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t ti = t + 4 * g + i;
      const bool use = ok && ti >= t_begin && ti < t_end;
      r.valid |= (uint32_t)use << (4 * s + i);
      vg[i] = use ? vg[i] : 0.0f;
      vs = use ? vs : vs & ~(0xFFu << (8 * i));
    }
    r.vs[s] = vs;
    r.vg[s] = vg;
  }
}

// NQ tiles of 16 query columns per wave; WQ = 4: the four waves of a workgroup
// hold different columns; WQ = 1: the same columns, and every fourth tile of
// the context each, joined in LDS at the end.
template <int D, int NQ, int WQ>
__global__ __launch_bounds__(256) void attention_kernel(AttnArgs a, int tiles_per_request) {
  constexpr int KF = D / 32, ND = D / 16, CT = 16 * NQ * WQ;
  __shared__ float s_o[WQ == 1 ? (ATT_WAVES - 1) * NQ * 16 * D : 1];
  __shared__ float s_ml[WQ == 1 ? ATT_WAVES * NQ * 16 * 2 : 1];
  const CacheArgs& cc = a.c;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int h = blockIdx.x % cc.H, split = blockIdx.y, G = a.G;   // a tile's KV heads are neighbours
  const int64_t tile_id = blockIdx.x / cc.H;

  // the request and the columns of this workgroup
  int64_t b = 0, ct = 0, q_begin = 0, q_len = 0;
  if (!cc.q_offsets) {
    b = tile_id / tiles_per_request;
    ct = tile_id - b * tiles_per_request;
    q_begin = b;
    q_len = 1;
  } else {
    int64_t base = 0;
    bool found = false;
    for (int64_t b0 = 0; b0 < cc.B && !found; b0 += 64) {
      const int64_t bb = b0 + lane;
      int64_t q0 = 0, n = 0;
      if (bb < cc.B) {
        q0 = cc.q_offsets[bb];
        const int64_t q1 = cc.q_offsets[bb + 1];
        n = q0 >= 0 && q1 <= a.T && q1 > q0 ? q1 - q0 : 0;
      }
      const int64_t mine = (n * G + CT - 1) / CT;
      int64_t incl = mine;
#pragma unroll
      for (int s = 1; s < 64; s *= 2) {
        const int64_t o = __shfl_up(incl, s, 64);
        if (lane >= s) incl += o;
      }
      const uint64_t hit = __ballot(base + incl > tile_id);
      if (hit) {
        const int src = __builtin_ctzll(hit);
        b = b0 + src;
        q_begin = __shfl(q0, src, 64);
        q_len = __shfl(n, src, 64);
        ct = tile_id - base - __shfl(incl - mine, src, 64);
        found = true;
      }
      base += __shfl(incl, 63, 64);
    }
    if (!found) return;                        // the grid is an upper bound
  }
  const int64_t L = cc.seq_lens[b];
  const int64_t col0 = ct * CT + (WQ == 1 ? 0 : wave * 16 * NQ);
  const int64_t ncols = q_len * G;

  // this wave's columns
  bool have[NQ];
  int64_t pos[NQ], row[NQ];                    // row: index of (token, head)
  f16x8 qf[NQ][KF];
  float colscale[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int64_t j = col0 + 16 * n + c;
    have[n] = j < ncols;
    const int64_t qi = have[n] ? j / G : 0, hg = have[n] ? j - qi * G : 0;
    pos[n] = have[n] ? L - q_len + qi : -1;
    const int64_t tq = q_begin + qi, head = (int64_t)h * G + hg;
    row[n] = tq * a.Hq + head;
    const uint16_t* qp = a.q + tq * a.q_token + head * a.q_head + g * (D / 4);
    uint4 w[KF];
    uint32_t amax = 0;
#pragma unroll
    for (int j2 = 0; j2 < KF; ++j2) {
      w[j2] = *reinterpret_cast<const uint4*>(qp + 8 * j2);
      amax = umax(amax, umax(umax(bf16x2_absmax_bits(w[j2].x), bf16x2_absmax_bits(w[j2].y)),
                             umax(bf16x2_absmax_bits(w[j2].z), bf16x2_absmax_bits(w[j2].w))));
    }
    amax = umax(amax, lane_xor_u32(amax, 16));
    amax = umax(amax, lane_xor_u32(amax, 32));
    const int e = amax ? 13 - ((int)(amax >> 7) - 127) : 0;
    colscale[n] = __builtin_ldexpf(a.scale_log2, -e);
#pragma unroll
    for (int j2 = 0; j2 < KF; ++j2) {
      const uint32_t ww[4] = {w[j2].x, w[j2].y, w[j2].z, w[j2].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qf[n][j2][2 * i] = (_Float16)__builtin_ldexpf(bf16_lo(ww[i]), e);
        qf[n][j2][2 * i + 1] = (_Float16)__builtin_ldexpf(bf16_hi(ww[i]), e);
      }
    }
  }

  // the tokens in reach of the wave's columns, as tiles [tile0, tile1) of this split
  const int64_t last = col0 + 16 * NQ < ncols ? col0 + 16 * NQ - 1 : ncols - 1;
  int64_t t_end = 0, t_begin = 0;
  if (col0 < ncols) {
    t_end = L - q_len + last / G + 1;
    const int64_t cap = cc.width << cc.P_log2;
    t_end = t_end > cap ? cap : t_end;
    t_begin = a.window ? L - q_len + col0 / G - a.window + 1 : 0;
    t_begin = t_begin < 0 ? 0 : t_begin;
  }
  int64_t tile0 = t_begin / TILE, tile1 = t_end > t_begin ? (t_end + TILE - 1) / TILE : tile0;
  {
    const int64_t per = (tile1 - tile0 + a.splits - 1) / a.splits;
    const int64_t lo = tile0 + per * split;
    tile1 = lo + per < tile1 ? lo + per : tile1;
    tile0 = lo;
  }

  f32x4 acc[NQ][ND];
  float m[NQ], l[NQ];
  int e_ref = -100;                            // Sref = 2^e_ref
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n] = NEG_INF;
    l[n] = 0.0f;
#pragma unroll
    for (int d = 0; d < ND; ++d) acc[n][d] = f32x4{0, 0, 0, 0};
  }

  RawTile<D> r;
  for (int64_t tile = tile0 + (WQ == 1 ? wave : 0); tile < tile1; tile += WQ == 1 ? ATT_WAVES : 1) {
    load_tile<D>(cc, b, h, tile * TILE, t_begin, t_end, c, g, r);

    // K to FP16
    f16x8 kf[2][KF];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      f16x2 sc[2] = {e4m3_pair<false>(r.ks[s]), e4m3_pair<true>(r.ks[s])};
#pragma unroll
      for (int j = 0; j < KF; ++j) {
        const int blk = j >> 1;                // of the lane's D / 64 blocks
        const _Float16 v = sc[blk >> 1][blk & 1];
        const f16x2 sv = {v, v};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f16x2 p = fp4_pair_at(r.k[s][j], i) * sv;
          kf[s][j][2 * i] = p.x;
          kf[s][j][2 * i + 1] = p.y;
        }
      }
    }
    // V to FP16: vf[d] holds the lane's value d of the tokens 4 g + i of both halves
    f16x8 vf[ND];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const f16x2 sc[2] = {e4m3_pair<false>(r.vs[s]), e4m3_pair<true>(r.vs[s])};
#pragma unroll
      for (int ip = 0; ip < 2; ++ip)
#pragma unroll
        for (int w = 0; w < (ND + 7) / 8; ++w) {
          const uint32_t ta = r.v[s][2 * ip][w], tb = r.v[s][2 * ip + 1][w];
          const uint32_t even = (ta & 0x0F0F0F0Fu) | ((tb << 4) & 0xF0F0F0F0u);
          const uint32_t odd = ((ta >> 4) & 0x0F0F0F0Fu) | (tb & 0xF0F0F0F0u);
#pragma unroll
          for (int d = 0; d < (ND < 8 ? ND : 8); ++d) {
            const f16x2 p = fp4_pair_at(d & 1 ? odd : even, d >> 1) * sc[ip];
            vf[8 * w + d][4 * s + 2 * ip] = p.x;
            vf[8 * w + d][4 * s + 2 * ip + 1] = p.y;
          }
        }
    }
    // Sref: a power of two above every second scale of V seen so far
    float smax = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) smax = fmaxf(smax, fmaxf(r.vg[0][i], r.vg[1][i]));
    smax = fmaxf(smax, __shfl_xor(smax, 16, 64));
    smax = fmaxf(smax, __shfl_xor(smax, 32, 64));
    const int e_new = max(e_ref, (int)(__float_as_uint(smax) >> 23) - 126);
    const float grow = __builtin_ldexpf(1.0f, e_ref - e_new);
    e_ref = e_new;
    f32x4 f[2];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) f[s][i] = __builtin_ldexpf(r.vg[s][i], 15 - e_ref);

#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      f32x4 x[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        x[s] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < KF; ++j) x[s] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[s][j], qf[n][j], x[s], 0, 0, 0);
      }
      const int64_t lo = a.window ? pos[n] - a.window : -1;
      float mx = m[n];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t t = r.t0 + 16 * s + 4 * g + i;
          const bool use = ((r.valid >> (4 * s + i)) & 1) && t <= pos[n] && t > lo;
          x[s][i] = use ? (x[s][i] * r.kg[s][i]) * colscale[n] : NEG_INF;
          mx = fmaxf(mx, x[s][i]);
        }
      mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
      mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
      const float mu = mx == NEG_INF ? 0.0f : mx;       // nothing in reach yet: every exponential is 0
      const float alpha = __builtin_amdgcn_exp2f(m[n] - mu);
      m[n] = mx;
      f16x8 wf;
      float sum = 0.0f;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = __builtin_amdgcn_exp2f(x[s][i] - mu);
          sum += p;
          wf[4 * s + i] = (_Float16)(p * f[s][i]);
        }
      l[n] = l[n] * alpha + sum;               // of this lane group's tokens
      const float scale = alpha * grow;
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        acc[n][d] *= scale;
        acc[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[d], wf, acc[n][d], 0, 0, 0);
      }
    }
  }

#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    l[n] += __shfl_xor(l[n], 16, 64);
    l[n] += __shfl_xor(l[n], 32, 64);
  }
  if (WQ == 1) {
    // join the four waves' tokens: the common maximum and sum first, then the
    // rows, each wave's brought to the common scale before it enters LDS
    if (g == 0)
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        s_ml[((wave * NQ + n) * 16 + c) * 2] = m[n];
        s_ml[((wave * NQ + n) * 16 + c) * 2 + 1] = l[n];
      }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float mw[ATT_WAVES], lw[ATT_WAVES], mx = NEG_INF;
#pragma unroll
      for (int w = 0; w < ATT_WAVES; ++w) {
        mw[w] = s_ml[((w * NQ + n) * 16 + c) * 2];
        lw[w] = s_ml[((w * NQ + n) * 16 + c) * 2 + 1];
        mx = fmaxf(mx, mw[w]);
      }
      const float mu = mx == NEG_INF ? 0.0f : mx;
      float lt = 0.0f;
#pragma unroll
      for (int w = 0; w < ATT_WAVES; ++w) lt += __builtin_amdgcn_exp2f(mw[w] - mu) * lw[w];
      const float f = lt > 0.0f ? __builtin_ldexpf(__builtin_amdgcn_exp2f(m[n] - mu) / lt, e_ref - 15) : 0.0f;
      m[n] = mx;
      l[n] = lt;
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        acc[n][d] *= f;
        if (wave > 0) *reinterpret_cast<f32x4*>(&s_o[((((wave - 1) * NQ + n) * ND + d) * 64 + lane) * 4]) = acc[n][d];
      }
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int w = 0; w < ATT_WAVES - 1; ++w)
          acc[n][d] += *reinterpret_cast<const f32x4*>(&s_o[(((w * NQ + n) * ND + d) * 64 + lane) * 4]);
  } else {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const float f = l[n] > 0.0f ? __builtin_ldexpf(1.0f / l[n], e_ref - 15) : 0.0f;
#pragma unroll
      for (int d = 0; d < ND; ++d) acc[n][d] *= f;
    }
  }

  // lane (c, g) holds, for its column, the values ND (4 g + i) + d
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    if (!have[n]) continue;
    const float lse2 = l[n] > 0.0f ? m[n] + __builtin_amdgcn_logf(l[n]) : NEG_INF;   // log2
    if (a.splits > 1) {
      const int64_t pr = (int64_t)split * a.T * a.Hq + row[n];
      if (g == 0) a.part_lse[pr] = lse2;
      if (l[n] > 0.0f)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int d = 0; d < ND; d += 4)
            *reinterpret_cast<f32x4*>(&a.part_o[pr * D + ND * (4 * g + i) + d]) =
                f32x4{acc[n][d][i], acc[n][d + 1][i], acc[n][d + 2][i], acc[n][d + 3][i]};
    } else {
      const int64_t tq = row[n] / a.Hq, head = row[n] - tq * a.Hq;
      uint16_t* o = a.out + tq * a.o_token + head * a.o_head;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int d = 0; d < ND; d += 4) {
          uint2 w;
          w.x = f32x2_to_bf16x2(acc[n][d][i], acc[n][d + 1][i]);
          w.y = f32x2_to_bf16x2(acc[n][d + 2][i], acc[n][d + 3][i]);
          *reinterpret_cast<uint2*>(o + ND * (4 * g + i) + d) = w;
        }
      if (a.lse && g == 0) a.lse[row[n]] = lse2 * 0.693147180559945309f;
    }
  }
}

// Joins the splits of one (token, head) per wave: weights 2^(lse_s - lse).
template <int D>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), rows = a.T * a.Hq;
  if (row >= rows) return;
  const int64_t tq = row / a.Hq, head = row - tq * a.Hq;
  if (request_of(a.c, tq) < 0) return;         // a row of no request is left as it was
  const float mine = lane < a.splits ? a.part_lse[lane * rows + row] : NEG_INF;
  float mx = mine;
#pragma unroll
  for (int s = 1; s < 64; s *= 2) mx = fmaxf(mx, __shfl_xor(mx, s, 64));
  const float e = mine == NEG_INF ? 0.0f : __builtin_amdgcn_exp2f(mine - mx);
  float total = e;
#pragma unroll
  for (int s = 1; s < 64; s *= 2) total += __shfl_xor(total, s, 64);
  float o[D / 64] = {};
  for (int s = 0; s < a.splits; ++s) {
    const float w = __shfl(e, s, 64);
    if (w == 0.0f) continue;                   // an empty split wrote no row
    const float* p = a.part_o + (s * rows + row) * D + lane * (D / 64);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) o[i] += w * p[i];
  }
  const float inv = total > 0.0f ? 1.0f / total : 0.0f;
  uint16_t* out = a.out + tq * a.o_token + head * a.o_head + lane * (D / 64);
#pragma unroll
  for (int i = 0; i < D / 64; ++i) out[i] = (uint16_t)f32x2_to_bf16x2(o[i] * inv, 0.0f);
  if (a.lse && lane == 0)
    a.lse[row] = total > 0.0f ? (mx + __builtin_amdgcn_logf(total)) * 0.693147180559945309f : NEG_INF;
}

template <int D>
static hipError_t launch_attention_d(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  const dim3 grid((unsigned)(a.c.H * p.tiles), (unsigned)p.splits);
  const int ct = 16 * p.nq * p.wq, tpr = (a.G + ct - 1) / ct;
  if (p.wq == 1) {
    if (p.nq == 1) hipLaunchKernelGGL((attention_kernel<D, 1, 1>), grid, dim3(256), 0, st, a, tpr);
    else hipLaunchKernelGGL((attention_kernel<D, D <= 128 ? 2 : 1, 1>), grid, dim3(256), 0, st, a, tpr);
  } else {
    hipLaunchKernelGGL((attention_kernel<D, D <= 128 ? 2 : 1, 4>), grid, dim3(256), 0, st, a, tpr);
  }
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && p.splits > 1) {
    hipLaunchKernelGGL(attention_join_kernel<D>, dim3((unsigned)((a.T * a.Hq + 3) / 4)), dim3(256), 0, st, a);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_attention(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  return a.c.D == 64 ? launch_attention_d<64>(a, p, st)
         : a.c.D == 128 ? launch_attention_d<128>(a, p, st) : launch_attention_d<256>(a, p, st);
}

}  // namespace mxq
