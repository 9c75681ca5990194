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
};

template <int BYTES>
__device__ __forceinline__ uint32_t load_small(const uint8_t* p) {
  if (BYTES == 1) return *p;
  if (BYTES == 2) return *reinterpret_cast<const uint16_t*>(p);
  return *reinterpret_cast<const uint32_t*>(p);
}

// The pages of a tile's halves (16 tokens lie in one page), -1 for none.
struct TilePages {
  int p[2];
};
__device__ __forceinline__ TilePages tile_pages(const CacheArgs& cc, const int32_t* table, int tile) {
  TilePages r;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int i = (tile * TILE + 16 * s) >> cc.P_log2;
    const int p = i < (int)cc.width ? table[i] : -1;
    r.p[s] = p < (int)cc.pages ? p : -1;
  }
  return r;
}

// Issues the loads of a tile; everything but the lane's offset inside the page
// is uniform over the wave.  A half without a page reads page 0.
template <int D>
__device__ __forceinline__ void load_tile(const CacheArgs& cc, const TilePages& tp, int h, int tile, int c, int g,
                                          RawTile<D>& r) {
  constexpr int VB = D / 32;                   // V bytes of a lane and token
  const int P = 1 << cc.P_log2;
  const uint32_t ko = c * (D / 2) + g * (D / 8), kso = c * (D / 16) + g * (D / 64);
  const uint32_t vo = 4 * g * (D / 2) + c * VB, vso = ((c * (D / 16) / 16) << cc.P_log2) + 4 * g;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int64_t page = tp.p[s] < 0 ? 0 : tp.p[s];
    const int slot = (tile * TILE + 16 * s) & (P - 1);
    const int64_t row = (int64_t)h * P + slot;
    const uint8_t* kc = cc.kc + page * cc.pc + row * (D / 2);
    if (D == 64) {
      const uint2 w = *reinterpret_cast<const uint2*>(kc + ko);
      r.k[s][0] = w.x, r.k[s][1] = w.y;
    } else {
#pragma unroll
      for (int j = 0; j < D / 128; ++j) {
        const uint4 w = *reinterpret_cast<const uint4*>(kc + ko + 16 * j);
        r.k[s][4 * j] = w.x, r.k[s][4 * j + 1] = w.y, r.k[s][4 * j + 2] = w.z, r.k[s][4 * j + 3] = w.w;
      }
    }
    r.ks[s] = load_small<D / 64>(cc.ks + page * cc.psc + row * (D / 16) + kso);
    const uint8_t* vc = cc.vc + page * cc.pc + row * (D / 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (VB == 8) {
        const uint2 w = *reinterpret_cast<const uint2*>(vc + vo + i * (D / 2));
        r.v[s][i][0] = w.x, r.v[s][i][(D + 127) / 128 - 1] = w.y;
      } else {
        r.v[s][i][0] = load_small<VB == 2 ? 2 : 4>(vc + vo + i * (D / 2));
      }
    }
    r.vs[s] = *reinterpret_cast<const uint32_t*>(cc.vs + page * cc.psc + (((int64_t)h * (D / 16)) << cc.P_log2) + slot +
                                                 vso);
    r.kg[s] = *reinterpret_cast<const f32x4*>(cc.kg + page * cc.pg + row + 4 * g);
    r.vg[s] = *reinterpret_cast<const f32x4*>(cc.vg + page * cc.pg + row + 4 * g);
  }
}

// Maximum over the lanes c, c + 16, c + 32, c + 48 (all four get it).
__device__ __forceinline__ float max_groups(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const float w = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const uint32_t x = __float_as_uint(w);
  const auto b = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// The columns of a wave: their statistics and output tiles.
template <int D, int NQ>
struct Columns {
  f16x8 q[NQ][D / 32];
  float cs[NQ];                 // logit (log2) per unit of q . k
  int pos[NQ], lo[NQ];          // tokens lo < t <= pos are in reach
  f32x4 acc[NQ][D / 16];
  float m[NQ], l[NQ];           // running maximum (of q . k), and this lane group's sum
  int e_ref;                    // Sref = 2^e_ref
};

// One tile.  `inside`: every token is in reach of every column.
template <int D, int NQ>
__device__ __forceinline__ void attend_tile(Columns<D, NQ>& o, RawTile<D>& r, const TilePages& tp, int tile,
                                            int t_begin, int t_end, bool inside, int g) {
  constexpr int KF = D / 32, ND = D / 16;
  if (!inside) {
    // a token outside the range, or without a page, may hold any bytes: its
    // V scales become zero here and its logit -inf below
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = tile * TILE + 16 * s + 4 * g + i;
        const bool use = tp.p[s] >= 0 && t >= t_begin && t < t_end;
        r.vg[s][i] = use ? r.vg[s][i] : 0.0f;
        r.vs[s] = use ? r.vs[s] : r.vs[s] & ~(0xFFu << (8 * i));
      }
  }
  // logits
  f32x4 x[NQ][2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const f16x2 sc[2] = {e4m3_pair<false>(r.ks[s]), e4m3_pair<true>(r.ks[s])};
#pragma unroll
    for (int n = 0; n < NQ; ++n) x[n][s] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < KF; ++j) {
      const int blk = j >> 1;                  // of the lane's D / 64 blocks
      const _Float16 v = sc[blk >> 1][blk & 1];
      const f16x2 sv = {v, v};
      f16x8 kf;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f16x2 p = fp4_pair_at(r.k[s][j], i) * sv;
        kf[2 * i] = p.x;
        kf[2 * i + 1] = p.y;
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n) x[n][s] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, o.q[n][j], x[n][s], 0, 0, 0);
    }
  }
  // Sref: a power of two above every second scale of V seen so far
  float smax = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) smax = fmaxf(smax, fmaxf(r.vg[0][i], r.vg[1][i]));
  smax = max_groups(smax);
  const int e_tile = __builtin_amdgcn_readfirstlane((int)(__float_as_uint(smax) >> 23) - 126);
  float grow = 1.0f;
  if (e_tile > o.e_ref) {
    grow = __builtin_ldexpf(1.0f, o.e_ref - e_tile);
    o.e_ref = e_tile;
  }
  f32x4 f[2];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) f[s][i] = __builtin_ldexpf(r.vg[s][i], 15 - o.e_ref);

  f16x8 wf[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    float mx = o.m[n];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[n][s][i] *= r.kg[s][i];
      if (!inside)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = tile * TILE + 16 * s + 4 * g + i;
          const bool use = tp.p[s] >= 0 && t <= o.pos[n] && t > o.lo[n];
          x[n][s][i] = use ? x[n][s][i] : NEG_INF;
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) mx = fmaxf(mx, x[n][s][i]);
    }
    mx = max_groups(mx);
    const float mu = mx == NEG_INF ? 0.0f : -mx * o.cs[n];   // nothing in reach yet: every exponential is 0
    if (__any(mx > o.m[n] || grow != 1.0f)) {
      const float alpha = __builtin_amdgcn_exp2f(__builtin_fmaf(o.m[n], o.cs[n], mu));
      const float scale = alpha * grow;
      o.l[n] *= alpha;
#pragma unroll
      for (int d = 0; d < ND; ++d) o.acc[n][d] *= scale;
    }
    o.m[n] = mx;
    float sum = 0.0f;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(x[n][s][i], o.cs[n], mu));
        sum += p;
        x[n][s][i] = p * f[s][i];
      }
    o.l[n] += sum;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const mxq_f32x2 pair = {x[n][s][i], x[n][s][i + 1]};
        const f16x2 hp = __builtin_convertvector(pair, f16x2);
        wf[n][4 * s + i] = hp.x;
        wf[n][4 * s + i + 1] = hp.y;
      }
  }
  // output: vf holds the lane's value d of the tokens 4 g + i of both halves
  uint32_t even[2][2][(ND + 7) / 8], odd[2][2][(ND + 7) / 8];
  f16x2 vsc[2][2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    vsc[s][0] = e4m3_pair<false>(r.vs[s]);
    vsc[s][1] = e4m3_pair<true>(r.vs[s]);
#pragma unroll
    for (int ip = 0; ip < 2; ++ip)
#pragma unroll
      for (int w = 0; w < (ND + 7) / 8; ++w) {
        const uint32_t ta = r.v[s][2 * ip][w], tb = r.v[s][2 * ip + 1][w];
        even[s][ip][w] = (ta & 0x0F0F0F0Fu) | ((tb << 4) & 0xF0F0F0F0u);
        odd[s][ip][w] = ((ta >> 4) & 0x0F0F0F0Fu) | (tb & 0xF0F0F0F0u);
      }
  }
#pragma unroll
  for (int d = 0; d < ND; ++d) {
    f16x8 vf;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int ip = 0; ip < 2; ++ip) {
        const f16x2 p = fp4_pair_at((d & 1 ? odd : even)[s][ip][d / 8], (d % 8) >> 1) * vsc[s][ip];
        vf[4 * s + 2 * ip] = p.x;
        vf[4 * s + 2 * ip + 1] = p.y;
      }
#pragma unroll
    for (int n = 0; n < NQ; ++n) o.acc[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, wf[n], o.acc[n][d], 0, 0, 0);
  }
}

// NQ tiles of 16 query columns per wave; WQ = 4: the four waves of a workgroup
// hold different columns; WQ = 1: the same columns, and every fourth tile of
// the context each, joined in LDS at the end.
template <int D, int NQ, int WQ>
__global__ __launch_bounds__(256, D <= 128 && NQ == 1 ? 3 : 2) void attention_kernel(AttnArgs a, int tiles_per_request) {
  constexpr int KF = D / 32, ND = D / 16, CT = 16 * NQ * WQ;
  __shared__ float s_o[WQ == 1 ? (ATT_WAVES - 1) * NQ * 16 * D : 1];
  __shared__ float s_ml[WQ == 1 ? ATT_WAVES * NQ * 16 * 2 : 1];
  const CacheArgs& cc = a.c;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int h = blockIdx.x % cc.H, split = blockIdx.y, G = a.G;   // a tile's KV heads are neighbours
  const int tile_id = blockIdx.x / cc.H;

  // the request and the columns of this workgroup
  int b = 0, ct = 0, q_begin = 0, q_len = 0;
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
      int q0 = 0, n = 0;
      if (bb < cc.B) {
        q0 = cc.q_offsets[bb];
        const int q1 = cc.q_offsets[bb + 1];
        n = q0 >= 0 && q1 <= a.T && q1 > q0 ? q1 - q0 : 0;
      }
      const int64_t mine = ((int64_t)n * G + CT - 1) / CT;
      int64_t incl = mine;
#pragma unroll
      for (int s = 1; s < 64; s *= 2) {
        const int64_t o = __shfl_up(incl, s, 64);
        if (lane >= s) incl += o;
      }
      const uint64_t hit = __ballot(base + incl > tile_id);
      if (hit) {
        const int src = __builtin_ctzll(hit);
        b = (int)b0 + src;
        q_begin = __shfl(q0, src, 64);
        q_len = __shfl(n, src, 64);
        ct = (int)(tile_id - base - __shfl(incl - mine, src, 64));
        found = true;
      }
      base += __shfl(incl, 63, 64);
    }
    if (!found) return;                        // the grid is an upper bound
    b = __builtin_amdgcn_readfirstlane(b);
    ct = __builtin_amdgcn_readfirstlane(ct);
    q_begin = __builtin_amdgcn_readfirstlane(q_begin);
    q_len = __builtin_amdgcn_readfirstlane(q_len);
  }
  const int L = max(cc.seq_lens[b], 0);
  const int32_t* table = cc.table + (int64_t)b * cc.ld_table;
  const int64_t col0 = (int64_t)ct * CT + (WQ == 1 ? 0 : wave * 16 * NQ);
  const int64_t ncols = (int64_t)q_len * G;

  // this wave's columns
  Columns<D, NQ> o;
  bool have[NQ];
  int64_t row[NQ];                             // index of (token, head)
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int64_t j = col0 + 16 * n + c;
    have[n] = j < ncols;
    const int qi = have[n] ? (int)(j / G) : 0, hg = have[n] ? (int)(j - (int64_t)qi * G) : 0;
    o.pos[n] = have[n] ? L - q_len + qi : -1;
    const int64_t lo = (int64_t)o.pos[n] - a.window;
    o.lo[n] = a.window && lo > -1 ? (int)lo : -1;
    const int64_t tq = (int64_t)q_begin + qi, head = (int64_t)h * G + hg;
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
    // the factor of a logit is kept positive (the maximum is taken before it
    // is applied): its sign goes to q, and where it vanishes, q does
    o.cs[n] = __builtin_ldexpf(fabsf(a.scale_log2), -e);
    float sign = a.scale_log2 < 0.0f ? -1.0f : 1.0f;
    if (!(o.cs[n] > 0.0f)) o.cs[n] = 1.0f, sign = 0.0f;
#pragma unroll
    for (int j2 = 0; j2 < KF; ++j2) {
      const uint32_t ww[4] = {w[j2].x, w[j2].y, w[j2].z, w[j2].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o.q[n][j2][2 * i] = (_Float16)(sign * __builtin_ldexpf(bf16_lo(ww[i]), e));
        o.q[n][j2][2 * i + 1] = (_Float16)(sign * __builtin_ldexpf(bf16_hi(ww[i]), e));
      }
    }
    o.m[n] = NEG_INF;
    o.l[n] = 0.0f;
#pragma unroll
    for (int d = 0; d < ND; ++d) o.acc[n][d] = f32x4{0, 0, 0, 0};
  }
  o.e_ref = -100;

  // the tokens in reach of the wave's columns, and those in reach of all of
  // them; as tiles, the part [tile0, tile1) of this split
  int t_end = 0, t_begin = 0, all_end = 0, all_begin = 0;
  if (col0 < ncols) {
    const int64_t last = col0 + 16 * NQ < ncols ? col0 + 16 * NQ - 1 : ncols - 1;
    const int64_t p0 = (int64_t)L - q_len + col0 / G, p1 = (int64_t)L - q_len + last / G;
    const int64_t cap = cc.width << cc.P_log2;
    const int64_t b0 = a.window ? p0 - a.window + 1 : 0, b1 = a.window ? p1 - a.window + 1 : 0;
    t_end = (int)(p1 + 1 > cap ? cap : p1 + 1);
    t_begin = (int)(b0 < 0 ? 0 : b0 > cap ? cap : b0);
    all_end = (int)(p0 + 1 > cap ? cap : p0 + 1);
    all_begin = (int)(b1 < 0 ? 0 : b1 > cap ? cap : b1);
  }
  int tile0 = t_begin / TILE, tile1 = t_end > t_begin ? (t_end + TILE - 1) / TILE : tile0;
  {
    const int per = (tile1 - tile0 + a.splits - 1) / a.splits;
    tile0 += per * split;
    tile1 = min(tile0 + per, tile1);
  }

  // a tile's loads are in flight while the one before it is computed, and the
  // page numbers of the next but one
  constexpr int STEP = WQ == 1 ? ATT_WAVES : 1;
  int tile = tile0 + (WQ == 1 ? wave : 0);
  if (tile < tile1) {
    RawTile<D> r[2];
    TilePages tp[2];
    tp[0] = tile_pages(cc, table, tile);
    tp[1] = tile_pages(cc, table, tile + STEP);
    load_tile<D>(cc, tp[0], h, tile, c, g, r[0]);
    while (true) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        // unconditional, so that the waits count them: behind the last tile
        // they read page 0, which stays unused
        const bool more = tile + STEP < tile1;
        if (!more) tp[1 - u].p[0] = tp[1 - u].p[1] = -1;
        load_tile<D>(cc, tp[1 - u], h, tile + STEP, c, g, r[1 - u]);
        const TilePages now = tp[u];
        tp[u] = tile_pages(cc, table, tile + 2 * STEP);
        const bool inside = tile * TILE >= all_begin && (tile + 1) * TILE <= all_end && now.p[0] >= 0 && now.p[1] >= 0;
        attend_tile<D, NQ>(o, r[u], now, tile, t_begin, t_end, inside, g);
        if (!more) goto done;
        tile += STEP;
      }
    }
  }
done:

  float m[NQ], l[NQ];                          // from here: the maximum as a logit (log2)
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n] = o.m[n] * o.cs[n];
    l[n] = o.l[n];
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
      const float f = lt > 0.0f ? __builtin_ldexpf(__builtin_amdgcn_exp2f(m[n] - mu) / lt, o.e_ref - 15) : 0.0f;
      m[n] = mx;
      l[n] = lt;
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        o.acc[n][d] *= f;
        if (wave > 0) *reinterpret_cast<f32x4*>(&s_o[((((wave - 1) * NQ + n) * ND + d) * 64 + lane) * 4]) = o.acc[n][d];
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
          o.acc[n][d] += *reinterpret_cast<const f32x4*>(&s_o[(((w * NQ + n) * ND + d) * 64 + lane) * 4]);
  } else {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const float f = l[n] > 0.0f ? __builtin_ldexpf(1.0f / l[n], o.e_ref - 15) : 0.0f;
#pragma unroll
      for (int d = 0; d < ND; ++d) o.acc[n][d] *= f;
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
                f32x4{o.acc[n][d][i], o.acc[n][d + 1][i], o.acc[n][d + 2][i], o.acc[n][d + 3][i]};
    } else {
      const int64_t tq = row[n] / a.Hq, head = row[n] - tq * a.Hq;
      uint16_t* out = a.out + tq * a.o_token + head * a.o_head;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int d = 0; d < ND; d += 4) {
          uint2 w;
          w.x = f32x2_to_bf16x2(o.acc[n][d][i], o.acc[n][d + 1][i]);
          w.y = f32x2_to_bf16x2(o.acc[n][d + 2][i], o.acc[n][d + 3][i]);
          *reinterpret_cast<uint2*>(out + ND * (4 * g + i) + d) = w;
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
