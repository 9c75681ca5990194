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
#include "mxq_kernels.h"

namespace mxq {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int FEW_WAVES = 4;                   // waves of a workgroup with few columns
constexpr int TILE = 32;                       // tokens of one step of a wave
constexpr float NEG_INF = -__builtin_inff();
// Exponentials are 2^(x - m + BASE) with x - m up to HEADROOM: an FP16 weight
// stays below 2^15, and below 2^-14 - BASE of the largest it loses bits.
constexpr float BASE = 10.0f, HEADROOM = 5.0f;

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

// What a wave reads of one 32-token tile: whole words (a narrower load is
// widened by the compiler as soon as it is issued, which waits for it), from
// which the lane shifts its share.
template <int D>
struct RawTile {
  uint32_t k[2][D / 32];        // [half][dword]: token c of the half, values g D / 4 + 8 j ..
  uint32_t ks[2];               // the word that holds its D / 64 block scales
  uint32_t v[2][4][(D + 127) / 128];   // [half][token 4 g + i]: the words that hold its D / 16 values
  uint32_t vs[2];               // block scales of those four tokens
  f32x4 kg[2], vg[2];           // second scales of those four tokens
};
// Shifts to the lane's block scales of K in their word (D / 64 bytes), and to
// its values of V (D = 64: half a word).
template <int D>
__device__ __forceinline__ int ks_shift(int g) { return D == 64 ? 8 * g : D == 128 ? 16 * (g & 1) : 0; }
template <int D>
__device__ __forceinline__ int v_shift(int c) { return D == 64 ? 16 * (c & 1) : 0; }

// Loads through a buffer descriptor: a uniform base, a uniform and a lane's
// 32-bit offset, so a load needs no address registers of its own.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, -1, 0x00020000);
}
__device__ __forceinline__ uint32_t load1(__amdgpu_buffer_rsrc_t b, uint32_t lane, uint32_t uniform) {
  return __builtin_amdgcn_raw_buffer_load_b32(b, lane, uniform, 0);
}
__device__ __forceinline__ uint2 load2(__amdgpu_buffer_rsrc_t b, uint32_t lane, uint32_t uniform) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(b, lane, uniform, 0));
}
__device__ __forceinline__ uint4 load4(__amdgpu_buffer_rsrc_t b, uint32_t lane, uint32_t uniform) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(b, lane, uniform, 0));
}

// A lane's offsets inside a 16-token half of a page.
template <int D>
struct LaneOffsets {
  uint32_t k, ks, v, vs, g;
  __device__ __forceinline__ LaneOffsets(const CacheArgs& cc, int c, int g_) {
    k = c * (D / 2) + g_ * (D / 8);
    ks = c * (D / 16) + (g_ * (D / 64) & ~3);
    v = 4 * g_ * (D / 2) + (c * (D / 32) & ~3);
    vs = ((c * (D / 16) / 16) << cc.P_log2) + 4 * g_;
    g = 16 * g_;
  }
};

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

// Issues the loads of a tile.  A half without a page reads page 0.
template <int D>
__device__ __forceinline__ void load_tile(const CacheArgs& cc, const TilePages& tp, int h, int tile,
                                          const LaneOffsets<D>& o, RawTile<D>& r) {
  const int P = 1 << cc.P_log2;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int64_t page = tp.p[s] < 0 ? 0 : tp.p[s];
    const uint32_t slot = (tile * TILE + 16 * s) & (P - 1);
    const int64_t head = (int64_t)h * P;
    const auto kc = buffer_at(cc.kc + page * cc.pc + head * (D / 2)), vc = buffer_at(cc.vc + page * cc.pc + head * (D / 2));
    const auto ks = buffer_at(cc.ks + page * cc.psc + head * (D / 16)), vs = buffer_at(cc.vs + page * cc.psc + head * (D / 16));
    const auto kg = buffer_at(cc.kg + page * cc.pg + head), vg = buffer_at(cc.vg + page * cc.pg + head);
    if (D == 64) {
      const uint2 w = load2(kc, o.k, slot * (D / 2));
      r.k[s][0] = w.x, r.k[s][1] = w.y;
    } else {
#pragma unroll
      for (int j = 0; j < D / 128; ++j) {
        const uint4 w = load4(kc, o.k + 16 * j, slot * (D / 2));
        r.k[s][4 * j] = w.x, r.k[s][4 * j + 1] = w.y, r.k[s][4 * j + 2] = w.z, r.k[s][4 * j + 3] = w.w;
      }
    }
    r.ks[s] = load1(ks, o.ks, slot * (D / 16));
    r.kg[s] = __builtin_bit_cast(f32x4, load4(kg, o.g, slot * 4));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (D == 256) {
        const uint2 w = load2(vc, o.v + i * (D / 2), slot * (D / 2));
        r.v[s][i][0] = w.x, r.v[s][i][(D + 127) / 128 - 1] = w.y;
      } else {
        r.v[s][i][0] = load1(vc, o.v + i * (D / 2), slot * (D / 2));
      }
    }
    r.vs[s] = load1(vs, o.vs, slot);
    r.vg[s] = __builtin_bit_cast(f32x4, load4(vg, o.g, slot * 4));
  }
}

// max without the quieting of signalling NaNs that fmaxf adds to values whose
// origin the compiler does not see
__device__ __forceinline__ float max2(float a, float b) {
  float r;
  asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
// Maximum over the lanes c, c + 16, c + 32, c + 48 (all four get it).
__device__ __forceinline__ float max_groups(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t x = __float_as_uint(max2(__uint_as_float(a[0]), __uint_as_float(a[1])));
  const auto b = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  return max2(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// Eight codes of K times their block scale sv.
__device__ __forceinline__ f16x8 k_fragment(uint32_t w, _Float16 scale) {
  const f16x2 sv = {scale, scale};
  f16x8 kf;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f16x2 p = fp4_pair_at(w, i) * sv;
    kf[2 * i] = p.x;
    kf[2 * i + 1] = p.y;
  }
  return kf;
}
// The even (odd) nibbles of two tokens' words side by side: byte i holds the
// value 2 i (2 i + 1) of token a, then of token b.
__device__ __forceinline__ uint32_t pair_nibbles(uint32_t a, uint32_t b, bool odd) {
  return odd ? ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u) : (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
}

// ------------------------------------------------------------------- work units
//
// A unit is a column tile of one request and a chunk of its context; a
// workgroup takes a unit for one KV head.  All chunks are about equally long
// (of all requests together, `target` of them), so that a batch of ragged
// lengths fills the chip evenly; with target 0 a request is one chunk.  The
// lengths are on the device: every workgroup finds its unit by scanning them.
struct Unit {
  int b, ct, chunk, chunks;     // request, column tile, chunk of its chunks
  int q_begin, q_len, L;
  int64_t base;                 // first unit of the request
};

struct RequestSize {
  int q_begin, q_len, L, cts, tiles;
};
__device__ __forceinline__ RequestSize request_size(const AttnArgs& a, int64_t b, int CT) {
  const CacheArgs& cc = a.c;
  RequestSize r = {0, 0, 0, 0, 0};
  if (b >= cc.B) return r;
  r.L = max(cc.seq_lens[b], 0);
  r.q_begin = (int)b;
  r.q_len = 1;
  if (cc.q_offsets) {
    r.q_begin = cc.q_offsets[b];
    const int end = cc.q_offsets[b + 1];
    r.q_len = r.q_begin >= 0 && end <= a.T && end > r.q_begin ? end - r.q_begin : 0;
  }
  r.cts = (int)(((int64_t)r.q_len * a.G + CT - 1) / CT);
  int64_t n = (int64_t)cc.width << cc.P_log2;
  n = n < r.L ? n : r.L;
  if (a.window && n > a.window + r.q_len) n = a.window + r.q_len;
  r.tiles = (int)((n + TILE - 1) / TILE);
  return r;
}

__device__ __forceinline__ int64_t wave_sum(int64_t v) {
#pragma unroll
  for (int s = 1; s < 64; s *= 2) v += __shfl_xor(v, s, 64);
  return v;
}

// False if the grid's unit u does not exist (the grid is an upper bound).
__device__ __forceinline__ bool find_unit(const AttnArgs& a, int u, int CT, int lane, Unit& out) {
  const int64_t B = a.c.B;
  RequestSize r = request_size(a, lane, CT);
  int chunk = 0x7FFFFFFF;
  if (a.target) {
    int64_t work = (int64_t)r.cts * r.tiles;
    for (int64_t b = 64 + lane; b < B; b += 64) {
      const RequestSize x = request_size(a, b, CT);
      work += (int64_t)x.cts * x.tiles;
    }
    work = wave_sum(work);
    const int64_t c = (work + a.target - 1) / a.target;
    chunk = (int)(c < MIN_CHUNK ? MIN_CHUNK : c > 0x7FFFFFFF ? 0x7FFFFFFF : c);
  }
  int64_t base = 0;
  for (int64_t b0 = 0; b0 < B; b0 += 64) {
    if (b0) r = request_size(a, b0 + lane, CT);
    const int chunks = r.tiles > chunk ? (r.tiles + chunk - 1) / chunk : 1;
    const int64_t mine = (int64_t)r.cts * chunks;
    int64_t incl = mine;
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
      const int64_t o = __shfl_up(incl, s, 64);
      if (lane >= s) incl += o;
    }
    const uint64_t hit = __ballot(base + incl > u);
    if (hit) {
      const int src = __builtin_ctzll(hit);
      out.b = __builtin_amdgcn_readfirstlane((int)b0 + src);
      out.base = base + __shfl(incl - mine, src, 64);
      out.chunks = __builtin_amdgcn_readlane(chunks, src);
      out.q_begin = __builtin_amdgcn_readlane(r.q_begin, src);
      out.q_len = __builtin_amdgcn_readlane(r.q_len, src);
      out.L = __builtin_amdgcn_readlane(r.L, src);
      const int i = __builtin_amdgcn_readfirstlane((int)(u - out.base));
      out.ct = i / out.chunks;
      out.chunk = i - out.ct * out.chunks;
      return true;
    }
    base += __shfl(incl, 63, 64);
  }
  return false;
}

// Tokens in reach of the columns [c0, c1) of a unit, and in reach of all of them.
struct Reach {
  int begin, end, all_begin, all_end;
};
__device__ __forceinline__ Reach reach(const AttnArgs& a, const Unit& u, int64_t c0, int64_t c1) {
  Reach r = {0, 0, 0, 0};
  const int64_t ncols = (int64_t)u.q_len * a.G;
  if (c1 > ncols) c1 = ncols;
  if (c0 >= c1) return r;
  const int64_t p0 = (int64_t)u.L - u.q_len + c0 / a.G, p1 = (int64_t)u.L - u.q_len + (c1 - 1) / a.G;
  const int64_t cap = a.c.width << a.c.P_log2;
  const int64_t b0 = a.window ? p0 - a.window + 1 : 0, b1 = a.window ? p1 - a.window + 1 : 0;
  auto clamp = [&](int64_t v) { return (int)(v < 0 ? 0 : v > cap ? cap : v); };
  r.end = clamp(p1 + 1);
  r.begin = clamp(b0);
  r.all_end = clamp(p0 + 1);
  r.all_begin = clamp(b1);
  return r;
}

// The tiles [first, second) of the unit's chunk.
__device__ __forceinline__ int2 chunk_tiles(const Unit& u, const Reach& r) {
  int t0 = r.begin / TILE, t1 = r.end > r.begin ? (r.end + TILE - 1) / TILE : t0;
  const int per = (t1 - t0 + u.chunks - 1) / u.chunks;
  t0 += per * u.chunk;
  return make_int2(t0, min(t0 + per, t1));
}

// ---------------------------------------------------------------------- columns

// The query columns of a wave and their running statistics.
template <int D, int NQ>
struct Columns {
  f16x8 q[NQ][D / 32];
  float cs[NQ];                 // logit (log2) per unit of q . k
  int pos[NQ], lo[NQ];          // tokens lo < t <= pos are in reach
  bool have[NQ];
  int64_t row[NQ];              // index of (token, head)
  f32x4 acc[NQ][D / 16];
  // m: the maximum the exponentials are taken against, as q . k; it moves when
  // a logit exceeds it by HEADROOM (log2), i.e. when q . k > limit.
  // mu = BASE - m cs
  float m[NQ], mu[NQ], limit[NQ];
  int e_ref;                    // Sref = 2^e_ref
};

template <int D, int NQ>
__device__ __forceinline__ void load_columns(const AttnArgs& a, const Unit& u, int h, int64_t col0, int c, int g,
                                             Columns<D, NQ>& o) {
  constexpr int KF = D / 32, ND = D / 16;
  const int64_t ncols = (int64_t)u.q_len * a.G;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int64_t j = col0 + 16 * n + c;
    o.have[n] = j < ncols;
    const int qi = o.have[n] ? (int)(j / a.G) : 0, hg = o.have[n] ? (int)(j - (int64_t)qi * a.G) : 0;
    o.pos[n] = o.have[n] ? u.L - u.q_len + qi : -1;
    const int64_t lo = (int64_t)o.pos[n] - a.window;
    o.lo[n] = a.window && lo > -1 ? (int)lo : -1;
    const int64_t tq = (int64_t)u.q_begin + qi, head = (int64_t)h * a.G + hg;
    o.row[n] = tq * a.Hq + head;
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
    o.limit[n] = NEG_INF;
    o.mu[n] = BASE;
#pragma unroll
    for (int d = 0; d < ND; ++d) o.acc[n][d] = f32x4{0, 0, 0, 0};
  }
  o.e_ref = -100;
}

// Masks the logits of a border tile.
template <int D, int NQ>
__device__ __forceinline__ void mask_logits(const Columns<D, NQ>& o, int n, f32x4* x, const TilePages& tp, int tile,
                                            int g) {
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int t0 = tile * TILE + 16 * s + 4 * g;
    const int last = tp.p[s] < 0 ? -1 : o.pos[n];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[s][i] = (t0 + i <= last) & (t0 + i > o.lo[n]) ? x[s][i] : NEG_INF;
  }
}

// A token outside [begin, end), or without a page, may hold any bytes: its V
// scales become zero (and its logit -inf).
__device__ __forceinline__ void drop_unused(f32x4* vg, uint32_t* vs, const TilePages& tp, int tile, int begin, int end,
                                            int g) {
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int t0 = tile * TILE + 16 * s + 4 * g;
    const int stop = tp.p[s] < 0 ? -1 : end;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool use = (t0 + i >= begin) & (t0 + i < stop);
      vg[s][i] = use ? vg[s][i] : 0.0f;
      vs[s] &= use ? 0xFFFFFFFFu : ~(0xFFu << (8 * i));
    }
  }
}

// Moves the maxima that a tile's logits x exceed by more than the headroom;
// returns whether the sums have to be rescaled, by alpha[n].
template <int D, int NQ>
__device__ __forceinline__ bool move_maxima(Columns<D, NQ>& o, const f32x4 (*x)[2], float* alpha) {
  bool over = false;
  float mx[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    mx[n] = x[n][0][0];
#pragma unroll
    for (int i = 1; i < 8; ++i) mx[n] = fmaxf(mx[n], x[n][i >> 2][i & 3]);
    over = over || mx[n] > o.limit[n];
  }
  if (!__any(over)) return false;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const float top = max2(o.m[n], max_groups(mx[n]));
    const float mu = top == NEG_INF ? BASE : BASE - top * o.cs[n];   // nothing in reach yet: every exponential is 0
    alpha[n] = __builtin_amdgcn_exp2f(__builtin_fmaf(o.m[n], o.cs[n], mu - BASE));
    o.m[n] = top;
    o.mu[n] = mu;
    o.limit[n] = top == NEG_INF ? NEG_INF : top + HEADROOM / o.cs[n];
  }
  return true;
}

// Writes the columns' rows (normalized, in acc) or the unit's partial rows.
// l: the sums against 2^(BASE - m cs).
template <int D, int NQ, int CT>
__device__ __forceinline__ void store_columns(const AttnArgs& a, const Unit& u, int64_t pu, int h, int col, int c, int g,
                                              const Columns<D, NQ>& o, const float* m, const float* l) {
  constexpr int ND = D / 16;
  // (no global store comes before this point: page numbers are read through
  // the scalar cache, which the compiler allows only to memory it sees untouched)
  if (u.ct == 0 && u.chunk == 0 && h == 0 && threadIdx.x == 0 && a.target)
    a.part_index[u.b] = make_int2((int)u.base, u.chunks);
  // lane (c, g) holds, for its column, the values ND (4 g + i) + d
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    if (!o.have[n]) continue;
    const float lse2 = l[n] > 0.0f ? m[n] - BASE + __builtin_amdgcn_logf(l[n]) : NEG_INF;   // log2
    if (u.chunks > 1) {
      const int64_t pr = pu * CT + col + 16 * n + c;
      if (g == 0) a.part_lse[pr] = lse2;
      if (l[n] > 0.0f)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int d = 0; d < ND; d += 4)
            *reinterpret_cast<f32x4*>(&a.part_o[pr * D + ND * (4 * g + i) + d]) =
                f32x4{o.acc[n][d][i], o.acc[n][d + 1][i], o.acc[n][d + 2][i], o.acc[n][d + 3][i]};
    } else {
      const int64_t tq = o.row[n] / a.Hq, head = o.row[n] - tq * a.Hq;
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
      if (a.lse && g == 0) a.lse[o.row[n]] = lse2 * 0.693147180559945309f;
    }
  }
}

// ------------------------------------------------------------- a few columns
//
// The four waves of a workgroup hold the same 16 NQ columns and take every
// fourth tile of the chunk each; they are joined in LDS.  Nothing is shared in
// between, so a wave dequantizes what it multiplies.

// One tile.  `inside`: every token is in reach of every column.
template <int D, int NQ>
__device__ __forceinline__ void attend_tile(Columns<D, NQ>& o, float* l, RawTile<D>& r, const TilePages& tp, int tile,
                                            int t_begin, int t_end, bool inside, int c, int g) {
  constexpr int KF = D / 32, ND = D / 16;
  if (!inside) {
    drop_unused(r.vg, r.vs, tp, tile, t_begin, t_end, g);
  }
  // logits
  f32x4 x[NQ][2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const uint32_t ks = r.ks[s] >> ks_shift<D>(g);
    const f16x2 sc[2] = {e4m3_pair<false>(ks), e4m3_pair<true>(ks)};
#pragma unroll
    for (int n = 0; n < NQ; ++n) x[n][s] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < KF; ++j) {
      const f16x8 kf = k_fragment(r.k[s][j], sc[j >> 2][(j >> 1) & 1]);   // block j / 2 of the lane's D / 64
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
  if (e_tile > o.e_ref) {
    const float grow = __builtin_ldexpf(1.0f, o.e_ref - e_tile);
    o.e_ref = e_tile;
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int d = 0; d < ND; ++d) o.acc[n][d] *= grow;
  }
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
#pragma unroll
    for (int s = 0; s < 2; ++s) x[n][s] *= r.kg[s];
    if (!inside) mask_logits(o, n, x[n], tp, tile, g);
  }
  float alpha[NQ];
  if (move_maxima(o, x, alpha))
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      l[n] *= alpha[n];
#pragma unroll
      for (int d = 0; d < ND; ++d) o.acc[n][d] *= alpha[n];
    }
  f32x4 f[2];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) f[s][i] = __builtin_ldexpf(r.vg[s][i], -o.e_ref);
  f16x8 wf[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(x[n][s][i], o.cs[n], o.mu[n]));
        l[n] += p;                             // of this lane group's tokens
        x[n][s][i] = p * f[s][i];
      }
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const mxq_f32x2 pair = {x[n][s][i], x[n][s][i + 1]};
        const f16x2 hp = __builtin_convertvector(pair, f16x2);
        wf[n][4 * s + i] = hp.x;
        wf[n][4 * s + i + 1] = hp.y;
      }
    }
  }
  // output: vf holds the lane's value d of the tokens 4 g + i of both halves
  const f16x2 vsc[2][2] = {{e4m3_pair<false>(r.vs[0]), e4m3_pair<true>(r.vs[0])},
                           {e4m3_pair<false>(r.vs[1]), e4m3_pair<true>(r.vs[1])}};
  uint32_t nib[2][2][2][(ND + 7) / 8];         // [odd][half][pair of tokens][word]
#pragma unroll
  for (int od = 0; od < 2; ++od)
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int ip = 0; ip < 2; ++ip)
#pragma unroll
        for (int w = 0; w < (ND + 7) / 8; ++w)
          nib[od][s][ip][w] =
              pair_nibbles(r.v[s][2 * ip][w] >> v_shift<D>(c), r.v[s][2 * ip + 1][w] >> v_shift<D>(c), od);
#pragma unroll
  for (int d = 0; d < ND; ++d) {
    f16x8 vf;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int ip = 0; ip < 2; ++ip) {
        const f16x2 p = fp4_pair_at(nib[d & 1][s][ip][d / 8], (d % 8) >> 1) * vsc[s][ip];
        vf[4 * s + 2 * ip] = p.x;
        vf[4 * s + 2 * ip + 1] = p.y;
      }
#pragma unroll
    for (int n = 0; n < NQ; ++n) o.acc[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, wf[n], o.acc[n][d], 0, 0, 0);
  }
}

template <int D, int NQ>
__global__ __launch_bounds__(256, D <= 128 && NQ == 1 ? 3 : 2) void attention_few_kernel(AttnArgs a) {
  constexpr int ND = D / 16, CT = 16 * NQ;
  __shared__ float s_o[(FEW_WAVES - 1) * CT * D];
  __shared__ float s_ml[FEW_WAVES * CT * 2];
  const CacheArgs& cc = a.c;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int h = blockIdx.x % cc.H, uid = blockIdx.x / cc.H;   // a unit's KV heads are neighbours
  Unit u;
  if (!find_unit(a, uid, CT, lane, u)) return;
  const int32_t* table = cc.table + (int64_t)u.b * cc.ld_table;
  const int64_t col0 = (int64_t)u.ct * CT;

  Columns<D, NQ> o;
  load_columns(a, u, h, col0, c, g, o);
  const Reach re = reach(a, u, col0, col0 + CT);
  const int2 tiles = chunk_tiles(u, re);
  float l[NQ] = {};

  // a tile's loads are in flight while the one before it is computed, and the
  // page numbers of the next but one
  int tile = tiles.x + wave;
  if (tile < tiles.y) {
    const LaneOffsets<D> off(cc, c, g);
    RawTile<D> r[2];
    TilePages tp[2];
    tp[0] = tile_pages(cc, table, tile);
    tp[1] = tile_pages(cc, table, tile + FEW_WAVES);
    load_tile<D>(cc, tp[0], h, tile, off, r[0]);
    while (true) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // unconditional, so that the waits count them: behind the last tile
        // they read page 0, which stays unused
        const bool more = tile + FEW_WAVES < tiles.y;
        if (!more) tp[1 - k].p[0] = tp[1 - k].p[1] = -1;
        load_tile<D>(cc, tp[1 - k], h, tile + FEW_WAVES, off, r[1 - k]);
        const TilePages now = tp[k];
        tp[k] = tile_pages(cc, table, tile + 2 * FEW_WAVES);
        const bool inside =
            tile * TILE >= re.all_begin && (tile + 1) * TILE <= re.all_end && now.p[0] >= 0 && now.p[1] >= 0;
        attend_tile<D, NQ>(o, l, r[k], now, tile, re.begin, re.end, inside, c, g);
        if (!more) goto done;
        tile += FEW_WAVES;
      }
    }
  }
done:

  // join the four waves' tokens: the common maximum and sum first, then the
  // rows, each wave's brought to the common scale before it enters LDS
  float m[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n] = o.m[n] * o.cs[n];                   // from here as a logit (log2)
    l[n] += __shfl_xor(l[n], 16, 64);
    l[n] += __shfl_xor(l[n], 32, 64);
    if (g == 0) {
      s_ml[((wave * NQ + n) * 16 + c) * 2] = m[n];
      s_ml[((wave * NQ + n) * 16 + c) * 2 + 1] = l[n];
    }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    float mw[FEW_WAVES], lw[FEW_WAVES], mx = NEG_INF;
#pragma unroll
    for (int w = 0; w < FEW_WAVES; ++w) {
      mw[w] = s_ml[((w * NQ + n) * 16 + c) * 2];
      lw[w] = s_ml[((w * NQ + n) * 16 + c) * 2 + 1];
      mx = fmaxf(mx, mw[w]);
    }
    const float top = mx == NEG_INF ? 0.0f : mx;
    float lt = 0.0f;
#pragma unroll
    for (int w = 0; w < FEW_WAVES; ++w) lt += __builtin_amdgcn_exp2f(mw[w] - top) * lw[w];
    const float f = lt > 0.0f ? __builtin_ldexpf(__builtin_amdgcn_exp2f(m[n] - top) / lt, o.e_ref) : 0.0f;
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
      for (int w = 0; w < FEW_WAVES - 1; ++w)
        o.acc[n][d] += *reinterpret_cast<const f32x4*>(&s_o[(((w * NQ + n) * ND + d) * 64 + lane) * 4]);
  store_columns<D, NQ, CT>(a, u, (int64_t)uid * cc.H + h, h, 0, c, g, o, m, l);
}

// -------------------------------------------------------------- many columns
//
// The W waves of a workgroup hold different columns and share the tiles: each
// tile's K and V are dequantized once, a share per wave, into LDS, as the
// very fragments the matrix instruction reads (a fragment is 64 lanes times 16
// bytes, written and read without bank conflicts).  LDS holds two phases of PH
// tiles: while one is attended to, the next one is filled, tile by tile, and
// a barrier separates them; inside a phase the waves drift apart, so that the
// matrix work of one meets the exponentials of another.  V carries its second
// scale here, V' = fp16(c fp16(s_b S_t 2^4 / Sref)), so that the weights are the
// plain exponentials.
constexpr int phase_tiles(int D) { return D <= 128 ? 4 : 2; }
template <int D>
constexpr int many_lds() { return 2 * phase_tiles(D) * ((D / 8) * 1024 + 128 + 4); }

template <int D, int W>
__global__ __launch_bounds__(64 * W, 2) void attention_many_kernel(AttnArgs a) {
  constexpr int KF = D / 32, ND = D / 16, NQ = D <= 128 ? 2 : 1, CT = 16 * NQ * W;
  constexpr int F = 2 * KF + ND;               // fragments of a tile
  static_assert(W == 8, "a word of V codes is eight values, one per wave");
  constexpr int PH = phase_tiles(D), SLOTS = 2 * PH;
  extern __shared__ uint4 s_frag[];            // [slot][F][64]
  f32x4* s_kg = reinterpret_cast<f32x4*>(s_frag + SLOTS * F * 64);   // [slot][8]: second scales of K
  int* s_e = reinterpret_cast<int*>(s_kg + SLOTS * 8);               // [slot]: exponent of Sref of V'
  const CacheArgs& cc = a.c;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int h = blockIdx.x % cc.H, uid = blockIdx.x / cc.H;
  Unit u;
  if (!find_unit(a, uid, CT, lane, u)) return;
  const int32_t* table = cc.table + (int64_t)u.b * cc.ld_table;
  const int64_t col_wg = (int64_t)u.ct * CT, col0 = col_wg + wave * 16 * NQ;

  Columns<D, NQ> o;
  load_columns(a, u, h, col0, c, g, o);
  float l[NQ] = {};
  const Reach wg = reach(a, u, col_wg, col_wg + CT), re = reach(a, u, col0, col0 + 16 * NQ);
  const int2 tiles = chunk_tiles(u, wg);
  const int P = 1 << cc.P_log2;

  // The wave's share of a tile, as loaded: KW fragments of K and VW of V.  Where
  // there are fewer than waves (D = 64) the lower half of the waves makes those
  // of K, the upper half those of V; every wave loads both, so that no load
  // depends on a branch.
  constexpr int KW = (2 * KF + W - 1) / W, VW = (ND + W - 1) / W;
  constexpr bool HALVES = F == W;
  const int first = HALVES ? wave % (W / 2) : wave;
  uint32_t kw[KW], ksc[KW], vw[VW][8];
  uint32_t vs[2];
  f32x4 kg[2], vg[2];
  const LaneOffsets<D> off(cc, c, g);
  auto load = [&](const TilePages& tp, int tile) {
    const int64_t head = (int64_t)h * P;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int64_t page = tp.p[s] < 0 ? 0 : tp.p[s];
      const uint32_t slot = (tile * TILE + 16 * s) & (P - 1);
      kg[s] = __builtin_bit_cast(f32x4, load4(buffer_at(cc.kg + page * cc.pg + head), off.g, slot * 4));
      vg[s] = __builtin_bit_cast(f32x4, load4(buffer_at(cc.vg + page * cc.pg + head), off.g, slot * 4));
      vs[s] = load1(buffer_at(cc.vs + page * cc.psc + head * (D / 16)), off.vs, slot);
      const auto vc = buffer_at(cc.vc + page * cc.pc + head * (D / 2));
#pragma unroll
      for (int k = 0; k < VW; ++k)             // fragment first + W k: value first of word k
#pragma unroll
        for (int i = 0; i < 4; ++i) vw[k][4 * s + i] = load1(vc, off.v + i * (D / 2), slot * (D / 2) + 4 * k);
    }
#pragma unroll
    for (int k = 0; k < KW; ++k) {
      const int id = first + W * k, s = id / KF;
      const int p = s ? tp.p[1] : tp.p[0];
      const int64_t page = p < 0 ? 0 : p;
      const uint32_t slot = (tile * TILE + 16 * s) & (P - 1);
      kw[k] = load1(buffer_at(cc.kc + page * cc.pc + head * (D / 2)), off.k, slot * (D / 2) + 4 * (id % KF));
      ksc[k] = load1(buffer_at(cc.ks + page * cc.psc + head * (D / 16)), off.ks, slot * (D / 16));
    }
  };
  int e_next = -100;                           // of the tile that was dequantized last
  auto dequantize = [&](const TilePages& tp, int tile, int slot) {
    const bool inside = tile * TILE >= wg.begin && (tile + 1) * TILE <= wg.end && tp.p[0] >= 0 && tp.p[1] >= 0;
    if (!inside) {
      drop_unused(vg, vs, tp, tile, wg.begin, wg.end, g);
    }
    float smax = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) smax = fmaxf(smax, fmaxf(vg[0][i], vg[1][i]));
    smax = max_groups(smax);
    e_next = max(e_next, __builtin_amdgcn_readfirstlane((int)(__float_as_uint(smax) >> 23) - 126));
    f16x2 sc[2][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const mxq_f32x2 b0 = __builtin_amdgcn_cvt_pk_f32_fp8(vs[s], false), b1 = __builtin_amdgcn_cvt_pk_f32_fp8(vs[s], true);
      const mxq_f32x2 p0 = {__builtin_ldexpf(b0.x * vg[s][0], 4 - e_next), __builtin_ldexpf(b0.y * vg[s][1], 4 - e_next)};
      const mxq_f32x2 p1 = {__builtin_ldexpf(b1.x * vg[s][2], 4 - e_next), __builtin_ldexpf(b1.y * vg[s][3], 4 - e_next)};
      sc[s][0] = __builtin_convertvector(p0, f16x2);
      sc[s][1] = __builtin_convertvector(p1, f16x2);
    }
    if (!HALVES || wave < W / 2)
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        const int id = first + W * k;
        const f16x8 fr = k_fragment(kw[k], e4m3_pair<false>(ksc[k] >> (ks_shift<D>(g) + 8 * (id % KF >> 1))).x);
        s_frag[(slot * F + id) * 64 + lane] = __builtin_bit_cast(uint4, fr);
      }
    if (!HALVES || wave >= W / 2)
#pragma unroll
      for (int k = 0; k < VW; ++k) {
        const int sh = 4 * first + v_shift<D>(c);
        f16x8 fr;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int ip = 0; ip < 2; ++ip) {
            // the pair's two codes into the low byte, whichever value of the word it is
            const uint32_t ta = vw[k][4 * s + 2 * ip] >> sh, tb = vw[k][4 * s + 2 * ip + 1] >> sh;
            const f16x2 p = fp4_pair<0>((ta & 15u) | ((tb & 15u) << 4)) * sc[s][ip];
            fr[4 * s + 2 * ip] = p.x;
            fr[4 * s + 2 * ip + 1] = p.y;
          }
        s_frag[(slot * F + 2 * KF + first + W * k) * 64 + lane] = __builtin_bit_cast(uint4, fr);
      }
    if (wave == 0 && c == 0) {
      s_kg[slot * 8 + g] = kg[0];
      s_kg[slot * 8 + 4 + g] = kg[1];
      if (g == 0) s_e[slot] = e_next;
    }
  };
  auto attend = [&](const TilePages& tp, int tile, int slot) {
    const bool inside = tile * TILE >= re.all_begin && (tile + 1) * TILE <= re.all_end && tp.p[0] >= 0 && tp.p[1] >= 0;
    // all of K's fragments are read before the first product and V's before the
    // exponentials, which cover their latency
    const uint4* frag = s_frag + slot * F * 64 + lane;
    uint4 fr[2 * KF > ND ? 2 * KF : ND];
#pragma unroll
    for (int j = 0; j < 2 * KF; ++j) fr[j] = frag[64 * j];
    const f32x4 kgs[2] = {s_kg[slot * 8 + g], s_kg[slot * 8 + 4 + g]};
    __builtin_amdgcn_sched_barrier(0);
    f32x4 x[NQ][2];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int n = 0; n < NQ; ++n) x[n][s] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < KF; ++j)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int n = 0; n < NQ; ++n)
          x[n][s] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, fr[s * KF + j]), o.q[n][j],
                                                           x[n][s], 0, 0, 0);
#pragma unroll
    for (int d = 0; d < ND; ++d) fr[d] = frag[64 * (2 * KF + d)];
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
      for (int s = 0; s < 2; ++s) x[n][s] *= kgs[s];
      if (!inside) mask_logits(o, n, x[n], tp, tile, g);
    }
    float alpha[NQ];
    if (move_maxima(o, x, alpha))
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        l[n] *= alpha[n];
#pragma unroll
        for (int d = 0; d < ND; ++d) o.acc[n][d] *= alpha[n];
      }
    f16x8 wf[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const mxq_f32x2 pair = {__builtin_amdgcn_exp2f(__builtin_fmaf(x[n][s][i], o.cs[n], o.mu[n])),
                                  __builtin_amdgcn_exp2f(__builtin_fmaf(x[n][s][i + 1], o.cs[n], o.mu[n]))};
          l[n] += pair.x + pair.y;             // of this lane group's tokens
          const f16x2 hp = __builtin_convertvector(pair, f16x2);
          wf[n][4 * s + i] = hp.x;
          wf[n][4 * s + i + 1] = hp.y;
        }
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      const f16x8 vf = __builtin_bit_cast(f16x8, fr[d]);
#pragma unroll
      for (int n = 0; n < NQ; ++n) o.acc[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, wf[n], o.acc[n][d], 0, 0, 0);
    }
  };

  if (tiles.x < tiles.y) {
    // `filled`: tiles dequantized so far; the loads of the next one are in
    // flight (behind the last tile they read some page, which stays unused)
    int filled = tiles.x;
    TilePages next = tile_pages(cc, table, filled);
    load(next, filled);
    auto fill = [&]() {
      const TilePages far = tile_pages(cc, table, filled + 1);
      dequantize(next, filled, (filled - tiles.x) % SLOTS);
      ++filled;
      next = far;
      load(next, filled);
    };
    for (int i = 0; i < PH && filled < tiles.y; ++i) fill();
    __syncthreads();
    TilePages now = tile_pages(cc, table, tiles.x);
    for (int tile = tiles.x; tile < tiles.y; ++tile) {
      const TilePages after = tile_pages(cc, table, tile + 1);
      const int slot = (tile - tiles.x) % SLOTS;
      // V' of this tile may be on a larger Sref than the sums
      const int e = __builtin_amdgcn_readfirstlane(s_e[slot]);
      if (e > o.e_ref) {
        const float grow = __builtin_ldexpf(1.0f, o.e_ref - e);
        o.e_ref = e;
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int d = 0; d < ND; ++d) o.acc[n][d] *= grow;
      }
      if (tile * TILE < re.end && (tile + 1) * TILE > re.begin) attend(now, tile, slot);
      if (filled < tiles.y) fill();
      if ((tile - tiles.x) % PH == PH - 1) __syncthreads();
      now = after;
    }
  }
  float m[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n] = o.m[n] * o.cs[n];
    l[n] += __shfl_xor(l[n], 16, 64);
    l[n] += __shfl_xor(l[n], 32, 64);
    const float f = l[n] > 0.0f ? __builtin_ldexpf(1.0f / l[n], o.e_ref - 4) : 0.0f;
#pragma unroll
    for (int d = 0; d < ND; ++d) o.acc[n][d] *= f;
  }
  store_columns<D, NQ, CT>(a, u, (int64_t)uid * cc.H + h, h, wave * 16 * NQ, c, g, o, m, l);
}

// Joins the chunks of one (token, head): weights 2^(lse_s - lse).  RW waves
// share a row's chunks (and meet in LDS): four where there are few rows, whose
// contexts are cut into many chunks then; eight chunks' rows are in flight.
template <int D, int RW>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a, int CT) {
  constexpr int DL = D / 64;                   // values of a lane
  __shared__ float s_o[RW > 1 ? 4 * 64 * DL : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, part = wave % RW;
  const int64_t row = ((int64_t)blockIdx.x * 4 + wave) / RW, rows = a.T * a.Hq;
  if (row >= rows) return;
  const int64_t tq = row / a.Hq, head = row - tq * a.Hq;
  const int64_t b = request_of(a.c, tq);
  if (b < 0) return;                           // a row of no request is left as it was
  const int2 ix = a.part_index[b];
  const int chunks = ix.y;
  if (chunks <= 1) return;                     // written by its only chunk
  const int h = (int)(head / a.G);
  const int64_t j = (tq - (a.c.q_offsets ? a.c.q_offsets[b] : tq)) * a.G + (head - (int64_t)h * a.G);
  const int64_t stride = (int64_t)a.c.H * CT;  // of a chunk
  const int64_t first = ((ix.x + j / CT * chunks) * a.c.H + h) * CT + j % CT;
  float mx = NEG_INF;
  for (int k = lane; k < chunks; k += 64) mx = fmaxf(mx, a.part_lse[first + k * stride]);
#pragma unroll
  for (int s = 1; s < 64; s *= 2) mx = fmaxf(mx, __shfl_xor(mx, s, 64));
  const float base = mx == NEG_INF ? 0.0f : mx;
  float total = 0.0f, o[DL] = {};
  for (int k0 = 0; k0 < chunks; k0 += 64) {
    const int n = min(chunks - k0, 64);
    const float e = lane < n ? a.part_lse[first + (k0 + lane) * stride] : NEG_INF;
    const float w = __builtin_amdgcn_exp2f(e - base);
    total += w;                                // of this lane's chunks
    for (int k = part; k < n; k += 8 * RW) {
      float v[8][DL], wk[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int kk = k + i * RW < n ? k + i * RW : part;   // behind the end: some chunk, with weight 0
        wk[i] = k + i * RW < n ? __shfl(w, kk, 64) : 0.0f;
        const float* po = a.part_o + (first + (k0 + kk) * stride) * D + lane * DL;
#pragma unroll
        for (int q = 0; q < DL; ++q) v[i][q] = po[q];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int q = 0; q < DL; ++q) o[q] += wk[i] > 0.0f ? wk[i] * v[i][q] : 0.0f;   // an empty chunk wrote no row
    }
  }
#pragma unroll
  for (int s = 1; s < 64; s *= 2) total += __shfl_xor(total, s, 64);
  if (RW > 1) {
#pragma unroll
    for (int q = 0; q < DL; ++q) s_o[(wave * DL + q) * 64 + lane] = o[q];
    __syncthreads();
    if (part) return;
#pragma unroll
    for (int q = 0; q < DL; ++q)
      for (int i = 1; i < RW; ++i) o[q] += s_o[((wave + i) * DL + q) * 64 + lane];
  }
  const float inv = total > 0.0f ? 1.0f / total : 0.0f;
  uint16_t* out = a.out + tq * a.o_token + head * a.o_head + lane * DL;
#pragma unroll
  for (int q = 0; q < DL; ++q) out[q] = (uint16_t)f32x2_to_bf16x2(o[q] * inv, 0.0f);
  if (a.lse && lane == 0)
    a.lse[row] = total > 0.0f ? (mx + __builtin_amdgcn_logf(total)) * 0.693147180559945309f : NEG_INF;
}

template <int D>
static hipError_t launch_attention_d(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  const dim3 grid((unsigned)(a.c.H * p.units));
  if (p.waves) {
    constexpr int lds = many_lds<D>();
    static std::atomic<uint32_t> done{0};
    hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(&attention_many_kernel<D, MANY_WAVES>), lds, done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((attention_many_kernel<D, MANY_WAVES>), grid, dim3(64 * MANY_WAVES), lds, st, a);
  } else if (p.nq == 1) {
    hipLaunchKernelGGL((attention_few_kernel<D, 1>), grid, dim3(256), 0, st, a);
  } else {
    if constexpr (D <= 128) hipLaunchKernelGGL((attention_few_kernel<D, 2>), grid, dim3(256), 0, st, a);
  }
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && p.target) {
    const int64_t rows = a.T * a.Hq;
    if (rows <= 4096)
      hipLaunchKernelGGL((attention_join_kernel<D, 4>), dim3((unsigned)rows), dim3(256), 0, st, a, p.ct);
    else
      hipLaunchKernelGGL((attention_join_kernel<D, 1>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, st, a, p.ct);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_attention(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  return a.c.D == 64 ? launch_attention_d<64>(a, p, st)
         : a.c.D == 128 ? launch_attention_d<128>(a, p, st) : launch_attention_d<256>(a, p, st);
}

}  // namespace mxq
