// Attention over an NVFP4 cache.
//
// For a query column (one token, one head): x_t = scale q . k_t over the
// context, o = sum_t softmax(x)_t v_t, with k_t = value(c) s_b S_t.  Computed in
// one pass over the cache with the running maximum m and sum l of the softmax.
//
// The products run on the FP16 matrix instructions.  value(c) s_b is an FP16
// number (at most six significant bits, 2^-10 .. 2688), so K's codes enter
// exactly; a query row is scaled by a power of two to have its largest element
// in [2^13, 2^14), which keeps its eight significant bits down to 2^-27 of that
// element.  S of K multiplies the logit, in binary32.  S of V is brought near
// one by Sref, a running power of two above every S_t seen.  With few columns it
// goes to the weights (fewer than the values), w_t = fp16(p_t S_t / Sref): one
// rounding, 2^-11 relative.  With many the dequantized tile is shared, and it goes
// to the values: fp16(p_t) meets fp16(c fp16(s_b S_t 2^4 / Sref)), three roundings,
// which keep the matrix instruction at FP16 and the weights free of a factor per
// token.  Below 2^-14 of the scale that a weight or value has, 2^-25 absolute takes
// the place of 2^-11.  Sums, maxima and logits are binary32, and l sums the
// exponentials before they are rounded.
//
// The ranges: q . k of the scaled row passes binary32 before the row's factor is
// applied, so keys must stay below 2^100 in magnitude; V rows below 2^-90 are not
// scaled up any further, and lose bits to FP16 (2^-124 of absolute error a token).
//
// What a column does not reach must not count, whatever it holds.  Its logit is
// replaced by -infinity; but V's values are shared by the columns of a tile, and
// 0 times NaN is NaN.  On border tiles, which hold tokens that some columns reach
// and others do not, S_t therefore goes to the weights of the columns that reach
// t, Sref is each column's own (a token 2^25 times larger than the others would
// push the weights of the rows before it out of FP16), and a NaN among a token's
// block scales is taken out of the shared values and put into S_t.
//
// Orientation: logits are computed transposed, X^T = K Q^T (A = tokens, B = query
// columns), and the output too, O^T = V^T W^T.  A lane then holds one column in
// both, so the softmax statistics and every rescaling are lane-local but for
// one exchange over the lane groups, and the weights W leave the first product
// in the register layout the second one reads: the order of the contracted
// tokens is permuted alike on both sides.  K's D values are contracted in the
// order the lanes hold them, q in the same; a pair of tokens' nibbles of V is
// interleaved so that one conversion gives two neighbouring contraction
// elements.
//
// Two kernels, by the query columns (row, head of the KV head's group) of a
// request, and a join where contexts are split.  With few columns the cache's
// bytes bound it, and the vector instructions that unpack them: 64 requests of up
// to 4096 tokens, 177 MB, 56.0 us (3.2 TB/s); four of up to 131071, 393 MB, 91 us
// (4.3 TB/s, a large copy has 4.8).  With
// many the matrix and vector units do: prompt chunks of 2048 rows behind 8192
// tokens, 437 GF, 791 us (553 TF/s).  A single short request is latency: 11.8
// us, the join's launch included.  Border tiles cost most where there is little
// else: four prompts of up to 512 tokens, 16 heads, 41.8 us (37.2 without what keeps
// their columns apart).  With head_dim 256 the kernel for many columns has more to
// hold than the registers do (q's fragments come back from scratch in the loop):
// chunks of 2048 rows behind 8192 tokens, 16 heads, 437 GF, 2057 us.

#include "cache_device.h"
#include "mxq_kernels.h"

namespace mxq {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

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

// What a lane takes of one 32-token tile: whole words, from which it shifts
// its share.
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

// The pages of a tile's halves (16 tokens lie in one page), -1 for none.
struct TilePages {
  int p[2];
};
// The table is read through the constant address space: the scalar cache
// then, whatever else the kernel stores (nothing writes the table meanwhile).
typedef const int32_t __attribute__((address_space(4))) * ScalarTable;
__device__ __forceinline__ ScalarTable scalar_table(const CacheArgs& cc, int b) {
  return (ScalarTable)(uintptr_t)(cc.table + (int64_t)b * cc.ld_table);
}
__device__ __forceinline__ TilePages tile_pages(const CacheArgs& cc, ScalarTable table, int tile) {
  TilePages r;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int i = (tile * TILE + 16 * s) >> cc.P_log2;
    const int p = i < (int)cc.width ? table[i] : -1;
    r.p[s] = p < (int)cc.pages ? p : -1;
  }
  return r;
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

// BASE less a maximum top (in units of cs): 0 for a column that has nothing in
// reach yet (every exponential is 0), NaN for a logit beyond binary32: against an
// infinite maximum every exponential would be 0, as if nothing were in reach.
__device__ __forceinline__ float base_less(float top, float cs) {
  const float r = top * cs;
  return top == NEG_INF ? BASE : fabsf(r) < __builtin_inff() ? BASE - r : __builtin_nanf("");
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
// workgroup takes a unit for one KV head.  All chunks are about equally long,
// of all requests together, so that a batch of ragged lengths fills the chip
// evenly; with target 0 a request is one chunk.  The
// lengths are on the device: every workgroup finds its unit by scanning them.
struct Unit {
  int b, ct, chunk, chunks;     // request, column tile, chunk of its chunks
  int q_begin, q_len, L;
  int base;                     // first unit of the request
};

struct RequestSize {
  int q_begin, q_len, L, cts, tiles;
};
__device__ __forceinline__ RequestSize request_size(const AttnArgs& a, int64_t b, int CT) {
  const CacheArgs& cc = a.c;
  RequestSize r = {0, 0, 0, 0, 0};
  if (b >= cc.B) return r;
  r.L = max(cc.seq_lens[b], 0);
  const RequestRows rows = request_rows(cc, b, a.T);
  r.q_begin = rows.begin;
  r.q_len = rows.len;
  r.cts = (int)(((int64_t)r.q_len * a.G + CT - 1) / CT);
  int64_t n = (int64_t)cc.width << cc.P_log2;
  n = n < r.L ? n : r.L;
  if (a.window && n > a.window + r.q_len) n = a.window + r.q_len;
  r.tiles = (int)((n + TILE - 1) / TILE);
  return r;
}

__device__ __forceinline__ float wave_sum(float v) {
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
    float work = (float)r.cts * (float)r.tiles;
    for (int64_t b = 64 + lane; b < B; b += 64) {
      const RequestSize x = request_size(a, b, CT);
      work += (float)x.cts * (float)x.tiles;
    }
    work = wave_sum(work);
    // never more than `target` chunks beside one per column tile (the grid's
    // bound; the sum is rounded, hence the margin); fewer, `coarse`, as long as
    // that leaves no chunk longer than LONG_CHUNK
    const float fine = work * (1.00001f / (float)a.target), coarse = work / (float)a.coarse;
    const float c = fmaxf(fine, fminf(coarse, (float)LONG_CHUNK));
    chunk = max(MIN_CHUNK, c < 1e9f ? (int)c + 1 : 0x7FFFFFFF);
  }
  int base = 0;
  for (int64_t b0 = 0; b0 < B; b0 += 64) {
    if (b0) r = request_size(a, b0 + lane, CT);
    const int chunks = r.tiles > chunk ? (r.tiles + chunk - 1) / chunk : 1;
    const int mine = r.cts * chunks;           // the host bounds the sum
    int incl = mine;
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
      const int o = __shfl_up(incl, s, 64);
      if (lane >= s) incl += o;
    }
    const uint64_t hit = __ballot(base + incl > u);
    if (hit) {
      const int src = __builtin_ctzll(hit);
      out.b = __builtin_amdgcn_readfirstlane((int)b0 + src);
      out.base = base + __builtin_amdgcn_readlane(incl - mine, src);
      out.chunks = __builtin_amdgcn_readlane(chunks, src);
      out.q_begin = __builtin_amdgcn_readlane(r.q_begin, src);
      out.q_len = __builtin_amdgcn_readlane(r.q_len, src);
      out.L = __builtin_amdgcn_readlane(r.L, src);
      const int i = __builtin_amdgcn_readfirstlane(u - out.base);
      out.ct = i / out.chunks;
      out.chunk = i - out.ct * out.chunks;
      return true;
    }
    base += __builtin_amdgcn_readlane(incl, 63);
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

// A query row in FP16: its elements times 2^e, the largest then in [2^13, 2^14).
// cs is the factor of a logit (log2) per unit of that product.  It is kept
// positive (maxima are taken before it is applied): its sign goes to q, and
// where it vanishes, q does.  A row with an infinity or a NaN becomes all NaN:
// logits of -infinity would look like tokens out of reach.
__device__ __forceinline__ int query_exponent(uint32_t amax, float scale_log2, float& cs, float& sign) {
  const int e = amax ? 13 - ((int)(amax >> 7) - 127) : 0;
  cs = __builtin_ldexpf(fabsf(scale_log2), -e);
  sign = scale_log2 < 0.0f ? -1.0f : 1.0f;
  if (!(cs > 0.0f)) cs = 1.0f, sign = 0.0f;
  if (amax >= 0x7F80u) sign = __builtin_nanf("");
  return e;
}
__device__ __forceinline__ f16x8 query_fragment(uint4 w, int e, float sign) {
  const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
  f16x8 q;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[2 * i] = (_Float16)(sign * __builtin_ldexpf(bf16_lo(ww[i]), e));
    q[2 * i + 1] = (_Float16)(sign * __builtin_ldexpf(bf16_hi(ww[i]), e));
  }
  return q;
}

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
  int e_ref[NQ];                // Sref = 2^e_ref
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
    float sign;
    const int e = query_exponent(amax, a.scale_log2, o.cs[n], sign);
#pragma unroll
    for (int j2 = 0; j2 < KF; ++j2) o.q[n][j2] = query_fragment(w[j2], e, sign);
    o.m[n] = NEG_INF;
    o.limit[n] = NEG_INF;
    o.mu[n] = BASE;
    o.e_ref[n] = -100;
#pragma unroll
    for (int d = 0; d < ND; ++d) o.acc[n][d] = f32x4{0, 0, 0, 0};
  }
}

// A border tile's logits and second scales of V as column n sees them.
template <int D, int NQ>
__device__ __forceinline__ void mask_column(const Columns<D, NQ>& o, int n, f32x4* x, f32x4* vg, const TilePages& tp,
                                            int tile, int g) {
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int t0 = tile * TILE + 16 * s + 4 * g;
    const int last = tp.p[s] < 0 ? -1 : o.pos[n];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool sees = (t0 + i <= last) & (t0 + i > o.lo[n]);
      x[s][i] = sees ? x[s][i] : NEG_INF;
      vg[s][i] = sees ? vg[s][i] : 0.0f;
    }
  }
}

// 0xFF in the bytes that are NaN as E4M3 numbers.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  const uint32_t m = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  return m | (m - (m >> 7));
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
    const float mu = base_less(top, o.cs[n]);
    alpha[n] = __builtin_amdgcn_exp2f(__builtin_fmaf(o.m[n], o.cs[n], mu - BASE));
    o.m[n] = top;
    o.mu[n] = mu;
    o.limit[n] = top == NEG_INF ? NEG_INF : top + HEADROOM / o.cs[n];
  }
  return true;
}

// Writes N neighbouring values of a column's normalized row, from value `at`
// on: to the output, or to the unit's partial row pr.
template <int D, int N>
__device__ __forceinline__ void store_run(const AttnArgs& a, const Unit& u, int64_t pr, int64_t row, int at,
                                          const float* v) {
  if (u.chunks > 1) {
    float* p = a.part_o + pr * D + at;
#pragma unroll
    for (int d = 0; d < N; d += 2) *reinterpret_cast<float2*>(p + d) = make_float2(v[d], v[d + 1]);
    return;
  }
  const int64_t tq = row / a.Hq, head = row - tq * a.Hq;
  uint16_t* out = a.out + tq * a.o_token + head * a.o_head + at;
#pragma unroll
  for (int d = 0; d < N; d += 2) *reinterpret_cast<uint32_t*>(out + d) = f32x2_to_bf16x2(v[d], v[d + 1]);
}
// The log sum of a column; m: its maximum as a logit (log2), l: its sum
// against 2^(BASE - m).  The sum is 0 exactly where nothing is in reach (the
// largest exponential is 2^BASE at least), and NaN where a logit is NaN: that
// stays NaN here, in the row and through the join.
__device__ __forceinline__ void store_lse(const AttnArgs& a, const Unit& u, int64_t pr, int64_t row, float m, float l) {
  const float lse2 = l == 0.0f ? NEG_INF : m - BASE + __builtin_amdgcn_logf(l);  // log2
  if (u.chunks > 1) a.part_lse[pr] = lse2;
  else if (a.lse) a.lse[row] = lse2 * 0.693147180559945309f;
}
// The join finds a request's units by this.
__device__ __forceinline__ void store_index(const AttnArgs& a, const Unit& u, int h) {
  if (a.target && u.ct == 0 && u.chunk == 0 && h == 0 && threadIdx.x == 0)
    a.part_index[u.b] = make_int2(u.base, u.chunks);
}

// ------------------------------------------------------- raw tiles through LDS
//
// A 32-token tile in LDS, as it is stored: codes [32, D / 2] of K, of V, scales
// [32, D / 16] of K, [D / 16, 32] of V, second scales of K, of V.  It is loaded by
// instructions that write LDS themselves, 1 KiB of codes or 64 words of scales
// each: neighbouring lanes read neighbouring bytes (as the operands of the
// matrix instruction lie in registers they would not), and no register waits.
template <int D>
struct RawLayout {
  static constexpr int CODES = 16 * D, KS = 2 * CODES, VS = KS + 2 * D, KG = VS + 2 * D, VG = KG + 128, SIZE = VG + 128;
  static constexpr int CODE_JOBS = 2 * D / 64, JOBS = CODE_JOBS + (D + 64) / 64;
};
// LDS row of V's row r: four neighbouring rows are rotated by r / 4, so that the
// lane groups, which read rows four apart, meet different banks.
__device__ __forceinline__ int v_row(int r) { return (r & ~3) | ((r + (r >> 2)) & 3); }
// Place of K's 16-byte piece q of row r, exchanged inside the row so that the
// same piece of 16 rows lies in different banks.
template <int D>
__device__ __forceinline__ int k_piece(int r, int q) { return q ^ ((r / (512 / D)) & (D / 32 - 1)); }

// A wave's part in loading the tiles: per lane a base address, and what a page
// and a token in it add to that.
struct TileLoad {
  const uint8_t* base;
  uint32_t page_stride, slot_stride;
  int half;                     // of the tile
  uint32_t lds;                 // uniform, inside the raw tile
};
template <int D>
__device__ __forceinline__ TileLoad tile_load(const CacheArgs& cc, int h, int job, int lane) {
  using Y = RawLayout<D>;
  const int64_t P = 1 << cc.P_log2;
  TileLoad t;
  if (job < Y::CODE_JOBS) {
    const bool v = job >= Y::CODE_JOBS / 2;
    const int q = v ? job - Y::CODE_JOBS / 2 : job;
    const int i = 64 * q + lane, at = i / (D / 32), chunk = i % (D / 32);
    const int r = v ? (at & ~3) | ((at - (at >> 2)) & 3) : at;  // the row that belongs there
    t.base = (v ? cc.vc : cc.kc) + (h * P + (r & 15)) * (D / 2) + 16 * (v ? chunk : k_piece<D>(r, chunk));
    t.page_stride = (uint32_t)cc.pc;
    t.slot_stride = D / 2;
    t.half = r >> 4;
    t.lds = (v ? Y::CODES : 0) + 1024 * q;
    return t;
  }
  const int q = job - Y::CODE_JOBS, w = 64 * q + lane;          // word w of the scales
  t.lds = Y::KS + 256 * q;
  t.page_stride = (uint32_t)cc.psc;
  if (w < D / 2) {
    const int r = w / (D / 64);
    t.base = cc.ks + (h * P + (r & 15)) * (D / 16) + 4 * (w % (D / 64));
    t.slot_stride = D / 16;
    t.half = r >> 4;
  } else if (w < D) {
    const int i = w - D / 2;
    t.base = cc.vs + ((int64_t)h * (D / 16) + (i >> 3)) * P + 4 * (i & 3);
    t.slot_stride = 1;
    t.half = (i >> 2) & 1;
  } else {
    const int i = w - D, r = i & 31;
    t.base = reinterpret_cast<const uint8_t*>((i < 32 ? cc.kg : cc.vg) + h * P + (r & 15));
    t.page_stride = (uint32_t)(4 * cc.pg);
    t.slot_stride = 4;
    t.half = r >> 4;
  }
  return t;
}
// Loads that write LDS at m0 + lane * size; no register receives them.
__device__ __forceinline__ void load_lds16(const void* p, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void load_lds4(const void* p, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(p), "{m0}"(lds) : "memory");
}
// ------------------------------------------------------------- a few columns
//
// The four waves of a workgroup hold the same 16 NQ columns and take every
// fourth tile of the chunk each; they are joined in LDS.  Nothing is shared in
// between, so a wave dequantizes what it multiplies, and a ring of raw tiles of
// its own, FEW_AHEAD of them in flight, needs no barrier.
constexpr int FEW_AHEAD = 1;
template <int D, int NQ>
constexpr int few_lds() {
  const int ring = FEW_WAVES * (FEW_AHEAD + 1) * RawLayout<D>::SIZE;
  const int join = ((FEW_WAVES - 1) * 16 * NQ * D + FEW_WAVES * 16 * NQ * 2) * 4;
  return ring > join ? ring : join;
}

// A lane's part of a raw tile in LDS.
template <int D>
__device__ __forceinline__ void read_tile(const uint8_t* raw, int c, int g, RawTile<D>& r) {
  using Y = RawLayout<D>;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int row = 16 * s + c;
    if (D == 64) {
      const uint2 w = *reinterpret_cast<const uint2*>(raw + row * 32 + 16 * k_piece<D>(row, g >> 1) + 8 * (g & 1));
      r.k[s][0] = w.x, r.k[s][1] = w.y;
    } else {
#pragma unroll
      for (int j = 0; j < D / 128; ++j) {
        const uint4 w = *reinterpret_cast<const uint4*>(raw + row * (D / 2) + 16 * k_piece<D>(row, g * (D / 128) + j));
        r.k[s][4 * j] = w.x, r.k[s][4 * j + 1] = w.y, r.k[s][4 * j + 2] = w.z, r.k[s][4 * j + 3] = w.w;
      }
    }
    r.ks[s] = *reinterpret_cast<const uint32_t*>(raw + Y::KS + row * (D / 16) + (g * (D / 64) & ~3));
    r.kg[s] = *reinterpret_cast<const f32x4*>(raw + Y::KG + 4 * (16 * s + 4 * g));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* v = raw + Y::CODES + v_row(16 * s + 4 * g + i) * (D / 2) + (c * (D / 32) & ~3);
      if (D == 256) {
        const uint2 w = *reinterpret_cast<const uint2*>(v);
        r.v[s][i][0] = w.x, r.v[s][i][(D + 127) / 128 - 1] = w.y;
      } else {
        r.v[s][i][0] = *reinterpret_cast<const uint32_t*>(v);
      }
    }
    r.vs[s] = *reinterpret_cast<const uint32_t*>(raw + Y::VS + (c * (D / 16) / 16) * 32 + 16 * s + 4 * g);
    r.vg[s] = *reinterpret_cast<const f32x4*>(raw + Y::VG + 4 * (16 * s + 4 * g));
  }
}

// One tile.  `inside`: every token is in reach of every column.
template <int D, int NQ>
__device__ __forceinline__ void attend_tile(Columns<D, NQ>& o, float* l, RawTile<D>& r, const TilePages& tp, int tile,
                                            bool inside, int c, int g) {
  constexpr int KF = D / 32, ND = D / 16;
  if (!inside) {
    // NaN block scales: the 16 lanes of a group hold the blocks of the same four tokens
    const uint32_t nan[2] = {nan_bytes(r.vs[0]), nan_bytes(r.vs[1])};
    if (__any((nan[0] | nan[1]) != 0))
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        r.vs[s] &= ~nan[s];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t hit = __ballot((nan[s] >> (8 * i) & 1) != 0);
          if (hit >> (16 * g) & 0xFFFF) r.vg[s][i] = __builtin_nanf("");
        }
      }
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
  f32x4 f[NQ][2];                              // the second scales of V, over Sref further down
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      x[n][s] *= r.kg[s];
      f[n][s] = r.vg[s];
    }
    if (!inside) mask_column(o, n, x[n], f[n], tp, tile, g);
  }
  // Sref: a power of two above every second scale of V that the column has seen so far
  int e_tile[NQ];
  bool grows = false;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    if (n > 0) e_tile[n] = e_tile[0];          // inside, all columns see the same tokens
    if (n == 0 || !inside) {
      float smax = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) smax = fmaxf(smax, fmaxf(f[n][0][i], f[n][1][i]));
      e_tile[n] = (int)(__float_as_uint(max_groups(smax)) >> 23) - 126;
    }
    grows = grows || e_tile[n] > o.e_ref[n];
  }
  if (__any(grows)) {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int e = max(o.e_ref[n], e_tile[n]);
      const float grow = __builtin_ldexpf(1.0f, o.e_ref[n] - e);
      o.e_ref[n] = e;
#pragma unroll
      for (int d = 0; d < ND; ++d) o.acc[n][d] *= grow;
    }
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
  for (int n = 0; n < NQ; ++n) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(x[n][s][i], o.cs[n], o.mu[n]));
        l[n] += p;                             // of this lane group's tokens
        x[n][s][i] = p * __builtin_ldexpf(f[n][s][i], -o.e_ref[n]);
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
  using Y = RawLayout<D>;
  constexpr int ND = D / 16, CT = 16 * NQ, SLOTS = FEW_AHEAD + 1;
  extern __shared__ __attribute__((aligned(16))) uint8_t s_few[];   // [waves][SLOTS] raw tiles; then the join
  float* s_ml = reinterpret_cast<float*>(s_few);
  float* s_o = s_ml + FEW_WAVES * CT * 2;
  const CacheArgs& cc = a.c;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int h = blockIdx.x % cc.H, uid = blockIdx.x / cc.H;   // a unit's KV heads are neighbours
  Unit u;
  if (!find_unit(a, uid, CT, lane, u)) return;
  const ScalarTable table = scalar_table(cc, u.b);
  const int64_t col0 = (int64_t)u.ct * CT;

  Columns<D, NQ> o;
  load_columns(a, u, h, col0, c, g, o);
  const Reach re = reach(a, u, col0, col0 + CT);
  const int2 tiles = chunk_tiles(u, re);
  float l[NQ] = {};

  if (tiles.x + wave < tiles.y) {
    TileLoad job[Y::JOBS];
#pragma unroll
    for (int k = 0; k < Y::JOBS; ++k) job[k] = tile_load<D>(cc, h, k, lane);
    const uint8_t* ring = s_few + wave * SLOTS * Y::SIZE;
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(ring);
    const int page_mask = (1 << cc.P_log2) - 1;
    uint32_t ok = 0;                           // halves with a page: two bits per tile in flight, the current lowest
    int ahead = tiles.x + wave;                // the tile to be issued next, and its pages
    TilePages pages = tile_pages(cc, table, ahead);
    // behind the last tile the loads read page 0, which stays unused, so that
    // the number in flight is always the same
    auto issue = [&](int slot, int behind) {
      TilePages tp = pages;
      if (ahead >= tiles.y) tp.p[0] = tp.p[1] = -1;
      ok |= (uint32_t)((tp.p[0] >= 0) | (tp.p[1] >= 0) << 1) << (2 * behind);
      const int p0 = max(tp.p[0], 0), p1 = max(tp.p[1], 0);
      const int s0 = (ahead * TILE) & page_mask, s1 = (ahead * TILE + 16) & page_mask;
      const uint32_t raw = lds0 + slot * Y::SIZE;
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");        // the slot's last readers have their values
#pragma unroll
      for (int k = 0; k < Y::JOBS; ++k) {
        const TileLoad& t = job[k];
        const uint8_t* p8 = t.base + (uint64_t)(uint32_t)(t.half ? p1 : p0) * t.page_stride +
                            (uint32_t)(t.half ? s1 : s0) * t.slot_stride;
        if (k < Y::CODE_JOBS) load_lds16(p8, raw + t.lds);
        else load_lds4(p8, raw + t.lds);
      }
      ahead += FEW_WAVES;
      pages = tile_pages(cc, table, ahead);
    };
#pragma unroll
    for (int i = 0; i < FEW_AHEAD; ++i) issue(i, i);
    int slot = 0;
    for (int tile = tiles.x + wave; tile < tiles.y; tile += FEW_WAVES) {
      issue(slot ? slot - 1 : FEW_AHEAD, FEW_AHEAD);
      asm volatile("s_waitcnt vmcnt(%0)" ::"i"(FEW_AHEAD * Y::JOBS) : "memory");
      RawTile<D> r;
      read_tile<D>(ring + slot * Y::SIZE, c, g, r);
      TilePages now;
      now.p[0] = ok & 1 ? 0 : -1;
      now.p[1] = ok & 2 ? 0 : -1;
      const bool inside = (tile * TILE >= re.all_begin) & ((tile + 1) * TILE <= re.all_end) & ((ok & 3) == 3);
      attend_tile<D, NQ>(o, l, r, now, tile, inside, c, g);
      ok >>= 2;
      slot = slot == FEW_AHEAD ? 0 : slot + 1;
    }
  }
  // the loads behind the last tile have landed in every wave's ring before it is used again
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

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
    const float f = lt == 0.0f ? 0.0f : __builtin_ldexpf(__builtin_amdgcn_exp2f(m[n] - top) / lt, o.e_ref[n]);
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
  store_index(a, u, h);
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    if (!o.have[n]) continue;
    const int64_t pr = ((int64_t)uid * cc.H + h) * CT + 16 * n + c;
    if (g == 0) store_lse(a, u, pr, o.row[n], m[n], l[n]);
    // lane (c, g) holds, for its column, the values ND (4 g + i) + d
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[ND];
#pragma unroll
      for (int d = 0; d < ND; ++d) v[d] = o.acc[n][d][i];
      store_run<D, ND>(a, u, pr, o.row[n], ND * (4 * g + i), v);
    }
  }
}

// -------------------------------------------------------------- many columns
//
// The eight waves of a workgroup hold 32 columns each and share the tiles.  A
// tile passes through LDS twice.  It arrives as it is stored, by loads that
// write LDS themselves (one or two instructions of a wave per tile, up to three
// phases ahead, which covers the latency of a page that no cache holds), and is
// then dequantized once, a share per wave, into the very fragments the matrix
// instruction reads (64 lanes times 16 bytes, no bank conflicts).  A phase is
// PH tiles: in phase p the waves attend to the fragments of p, make those of
// p + 1 and issue the loads of p + 3; one barrier ends it.  Of the two waves of
// a SIMD one attends first and the other fills first, so that one's matrix
// work meets the other's conversions.
//
// The 32x32x16 instruction takes 32 tokens and 32 columns at a time: half the
// instructions of the 16x16x32 form, and a lane holds one column.  Lane (c, hh)
// = (lane % 32, lane / 32): for K token c, the D / 2 values from hh D / 2 on; for
// V the D / 32 values from c D / 32 on of the tokens 16 kk + 4 hh + i and
// 16 kk + 8 + 4 hh + i (i < 4), kk = 0, 1.  V carries its second scale here, V' =
// fp16(c fp16(s_b S_t 2^4 / Sref)), so that the weights are the plain
// exponentials.
//
// That holds for the whole tiles, whose tokens all columns of the workgroup
// reach.  The others, the border tiles, have fragments of c s_b 2^4 (exact), and
// S_t goes to the weights (a second rounding of those), over a Sref of the column,
// 2^bump times the shared one.
template <int D>
struct ManyLayout {
  static constexpr int W = MANY_WAVES, CT = 32 * W;
  static constexpr int PH = D <= 128 ? 2 : 1, RING = 4;         // tiles of a phase, phases of raw tiles
  static constexpr int NK = D / 16, NV = D / 16, F = NK + NV;   // fragments of a tile
  using Raw = RawLayout<D>;
  static constexpr int CODES = Raw::CODES, KS = Raw::KS, VS = Raw::VS, KG = Raw::KG, VG = Raw::VG, RAW = Raw::SIZE;
  static constexpr int RAW0 = 2 * PH * F * 1024, LDS = RAW0 + RING * PH * RAW;
  static constexpr int CODE_JOBS = Raw::CODE_JOBS, JOBS = Raw::JOBS, JW = (JOBS + W - 1) / W;   // JW: of a wave
};
// Waits until at most N of the wave's loads are in flight and for its LDS
// accesses, then for the workgroup.
template <int N>
__device__ __forceinline__ void loads_barrier() {
  static_assert(N < 64, "vmcnt");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"(N) : "memory");
}

template <int D>
__global__ __launch_bounds__(64 * MANY_WAVES, 2) void attention_many_kernel(AttnArgs a) {
  using Y = ManyLayout<D>;
  constexpr int W = Y::W, PH = Y::PH, NK = Y::NK, NV = Y::NV, F = Y::F, DT = D / 32;
  extern __shared__ __attribute__((aligned(16))) uint8_t s_many[];
  const CacheArgs& cc = a.c;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 31, hh = lane >> 5;
  const int h = blockIdx.x % cc.H, uid = blockIdx.x / cc.H;
  Unit u;
  if (!find_unit(a, uid, Y::CT, lane, u)) return;
  const ScalarTable table = scalar_table(cc, u.b);
  const int64_t col_wg = (int64_t)u.ct * Y::CT, col0 = col_wg + wave * 32, ncols = (int64_t)u.q_len * a.G;
  const Reach wg = reach(a, u, col_wg, col_wg + Y::CT), re = reach(a, u, col0, col0 + 32);
  const int2 tiles = chunk_tiles(u, wg);
  const int count = tiles.y - tiles.x;
  const int w0 = (wg.all_begin + TILE - 1) / TILE, w1 = wg.all_end / TILE;   // the whole tiles
  auto is_whole = [&](int tile, int valid) { return (tile >= w0) & (tile < w1) & (valid == 3); };
  // phases of whole tiles only, but for missing pages
  const int pw0 = (max(w0 - tiles.x, 0) + PH - 1) / PH, pw1 = (min(w1, tiles.y) - tiles.x) / PH;

  // loads: phase p into ring slot p % RING
  // (a wave without a load of its own repeats the last one, the same bytes to
  // the same place, so that every wave has JW in flight per tile)
  TileLoad job[Y::JW];
#pragma unroll
  for (int k = 0; k < Y::JW; ++k) job[k] = tile_load<D>(cc, h, min(wave + W * k, Y::JOBS - 1), lane);
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(s_many);
  // which halves of the tiles have a page: two bits per tile, the current phase lowest
  uint32_t ok = 0;
  TilePages pages[PH];                         // of the phase to be issued next
  auto look_up = [&](int p) {
#pragma unroll
    for (int i = 0; i < PH; ++i) pages[i] = tile_pages(cc, table, tiles.x + p * PH + i);
  };
  look_up(0);
  const int page_mask = (1 << cc.P_log2) - 1;
  auto issue = [&](int p, int ahead) {
#pragma unroll
    for (int i = 0; i < PH; ++i) {
      const int tile = tiles.x + p * PH + i;
      TilePages tp = pages[i];
      if (p * PH + i >= count) tp.p[0] = tp.p[1] = -1;          // keeps the number of loads in flight
      ok |= (uint32_t)((tp.p[0] >= 0) | (tp.p[1] >= 0) << 1) << (2 * (ahead * PH + i));
      const int p0 = max(tp.p[0], 0), p1 = max(tp.p[1], 0);
      const int s0 = (tile * TILE) & page_mask, s1 = (tile * TILE + 16) & page_mask;
      const uint32_t raw = lds0 + Y::RAW0 + ((p & (Y::RING - 1)) * PH + i) * Y::RAW;
#pragma unroll
      for (int k = 0; k < Y::JW; ++k) {
        const TileLoad& t = job[k];
        const uint8_t* p8 = t.base + (uint64_t)(uint32_t)(t.half ? p1 : p0) * t.page_stride +
                            (uint32_t)(t.half ? s1 : s0) * t.slot_stride;
        if (wave + W * k < Y::CODE_JOBS) load_lds16(p8, raw + t.lds);
        else load_lds4(p8, raw + t.lds);
      }
    }
    look_up(p + 1);
  };

  // columns: lane (c, hh) holds column col0 + c; values hh D / 2 + 8 j of q
  const bool have = col0 + c < ncols;
  const int qi = have ? (int)((col0 + c) / a.G) : 0, hg = have ? (int)(col0 + c - (int64_t)qi * a.G) : 0;
  const int pos = have ? u.L - u.q_len + qi : -1;
  const int64_t low = (int64_t)pos - a.window;
  const int lo = a.window && low > -1 ? (int)low : -1;
  const int64_t tq = (int64_t)u.q_begin + qi, head = (int64_t)h * a.G + hg, row = tq * a.Hq + head;
  f16x8 q[NK];
  float cs;
  {
    const uint16_t* qp = a.q + tq * a.q_token + head * a.q_head + hh * (D / 2);
    uint4 w[NK];
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      w[j] = *reinterpret_cast<const uint4*>(qp + 8 * j);
      amax = umax(amax, umax(umax(bf16x2_absmax_bits(w[j].x), bf16x2_absmax_bits(w[j].y)),
                             umax(bf16x2_absmax_bits(w[j].z), bf16x2_absmax_bits(w[j].w))));
    }
    amax = umax(amax, lane_xor_u32(amax, 32));
    float factor;
    const int e = query_exponent(amax, a.scale_log2, cs, factor);
#pragma unroll
    for (int j = 0; j < NK; ++j) q[j] = query_fragment(w[j], e, factor);
  }
  issue(0, 0);
  issue(1, 1);
  issue(2, 2);
  f32x16 acc[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) acc[d] = f32x16{};
  float m = NEG_INF, limit = NEG_INF, mu = BASE, l = 0.0f;
  int e_ref = -100, e_fill = -100;             // exponents of Sref: of the sums, of the fragments made last
  int bump = 0;                                // the column's sums are on 2^(e_ref + bump)
  bool bumped = false, apart = false;          // a column of the wave has a bump; has one and meets whole tiles
  bool whole_now = false, whole_next = false;  // this phase, the next one: whole tiles only

  // ranges of tiles: some token in reach of the wave's columns, every token in reach of all of them
  const int any0 = re.begin / TILE, any1 = (re.end + TILE - 1) / TILE;
  const int all0 = (re.all_begin + TILE - 1) / TILE, all1 = re.all_end / TILE;

  // The exponent of Sref for phase p, whose tiles are there: a power of two
  // above every second scale of V in the whole tiles so far.  In a border tile, a
  // token with a NaN among its block scales gets a NaN for S: the fragments go
  // without the NaN (all waves write the same, for attend alone).
  auto scale_of = [&](int p, int shift) {
    constexpr uint32_t ALL = (1u << (2 * PH)) - 1;
    whole_next = (p >= pw0) & (p < pw1) & ((ok >> (2 * PH * shift) & ALL) == ALL);
    const int h2 = PH == 2 ? hh : 0;
    float v = reinterpret_cast<const float*>(s_many + Y::RAW0 + ((p & (Y::RING - 1)) * PH + h2) * Y::RAW + Y::VG)[c];
    if (__builtin_expect(!whole_next, 0)) {
#pragma unroll
      for (int i = 0; i < PH; ++i) {
        if (is_whole(tiles.x + p * PH + i, (int)(ok >> (2 * (shift * PH + i))) & 3)) continue;
        if (PH == 1 || hh == i) v = 0.0f;
        uint8_t* raw = s_many + Y::RAW0 + ((p & (Y::RING - 1)) * PH + i) * Y::RAW;
#pragma unroll
        for (int w = 0; w < (D + 127) / 128; ++w) {
          const int at = (64 * w + lane) & (D / 2 - 1);         // word: block at / 8, tokens 4 (at % 8) ..
          const uint32_t nan = nan_bytes(*reinterpret_cast<const uint32_t*>(raw + Y::VS + 4 * at));
          if (nan)
#pragma unroll
            for (int t = 0; t < 4; ++t)
              if (nan >> (8 * t) & 1) reinterpret_cast<float*>(raw + Y::VG)[4 * (at & 7) + t] = __builtin_nanf("");
        }
      }
    }
    e_fill = max(e_fill, (int)(wave_max_u32(__float_as_uint(v)) >> 23) - 126);
  };

  // Makes the fragments of tile i of phase p.
  auto fill = [&](int p, int i, int shift) {
    const int tile = tiles.x + p * PH + i, valid = (int)(ok >> (2 * (shift * PH + i))) & 3;
    const uint8_t* raw = s_many + Y::RAW0 + ((p & (Y::RING - 1)) * PH + i) * Y::RAW;
    uint4* frag = reinterpret_cast<uint4*>(s_many) + ((p & 1) * PH + i) * F * 64 + lane;
    const bool whole = whole_next || is_whole(tile, valid);
    const float to_ref = __builtin_ldexpf(1.0f, whole ? 4 - e_fill : 4);
    // K: fragment j holds the values hh D / 2 + 8 j of token c
    const int kfirst = NK >= W ? wave : wave % NK;
    if (NK >= W || wave < NK)
#pragma unroll
      for (int k = 0; k < (NK + W - 1) / W; ++k) {
        const int j = kfirst + W * k, word = hh * NK + j;       // of the token's codes
        const uint32_t code =
            *reinterpret_cast<const uint32_t*>(raw + c * (D / 2) + 16 * k_piece<D>(c, word >> 2) + 4 * (word & 3));
        const uint32_t sc = raw[Y::KS + c * (D / 16) + (word >> 1)];
        frag[64 * j] = __builtin_bit_cast(uint4, k_fragment(code, e4m3_pair<false>(sc).x));
      }
    if (NV >= W || wave >= NK)
#pragma unroll
      for (int k = 0; k < (NV + W - 1) / W; ++k) {
        const int v = (NV >= W ? wave : wave - NK) + W * k, dt = v % DT, kk = v / DT;
        const uint8_t* codes = raw + Y::CODES + (c * DT / 8) * 4;
        const int sh = 4 * ((c * DT + dt) & 7);
        f16x8 fr;
#pragma unroll
        for (int b = 0; b < 2; ++b) {          // tokens r .. r + 3
          const int r = 16 * kk + 8 * b + 4 * hh;
          f32x4 vg = *reinterpret_cast<const f32x4*>(raw + Y::VG + 4 * r);
          uint32_t vs = *reinterpret_cast<const uint32_t*>(raw + Y::VS + (c * DT / 16) * 32 + r);
          if (__builtin_expect(!whole, 0)) {
            vg = f32x4{1, 1, 1, 1};
            vs &= ~nan_bytes(vs);
          }
          uint32_t w[4];
#pragma unroll
          for (int t = 0; t < 4; ++t)
            w[t] = (*reinterpret_cast<const uint32_t*>(codes + v_row(r + t) * (D / 2)) >> sh) & 15u;
          // the conversion applies the power of two; the factor of a border tile is exact
          const mxq_f32x2 b0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(vs, to_ref, false);
          const mxq_f32x2 b1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(vs, to_ref, true);
          const mxq_f32x2 f0 = {b0.x * vg[0], b0.y * vg[1]}, f1 = {b1.x * vg[2], b1.y * vg[3]};
          const f16x2 p0 = fp4_pair<0>(w[0] | w[1] << 4) * __builtin_convertvector(f0, f16x2);
          const f16x2 p1 = fp4_pair<0>(w[2] | w[3] << 4) * __builtin_convertvector(f1, f16x2);
          fr[4 * b] = p0.x, fr[4 * b + 1] = p0.y, fr[4 * b + 2] = p1.x, fr[4 * b + 3] = p1.y;
        }
        frag[64 * (NK + v)] = __builtin_bit_cast(uint4, fr);
      }
  };

  auto attend = [&](int p, int i) {
    const int tile = tiles.x + p * PH + i, valid = (int)(ok >> (2 * i)) & 3;
    if ((tile < any0) | (tile >= any1) | (p * PH + i >= count)) return;
    const uint4* frag = reinterpret_cast<const uint4*>(s_many) + ((p & 1) * PH + i) * F * 64 + lane;
    const uint8_t* raw = s_many + Y::RAW0 + ((p & (Y::RING - 1)) * PH + i) * Y::RAW;
    // fragments are read eight at a time, V's first ones before the
    // exponentials, which cover their latency
    uint4 fr[8];
    f32x16 x = {};
#pragma unroll
    for (int j0 = 0; j0 < NK; j0 += 8) {
#pragma unroll
      for (int j = 0; j < 8 && j < NK; ++j) fr[j] = frag[64 * (j0 + j)];
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < 8 && j < NK; ++j)
        x = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, fr[j]), q[j0 + j], x, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < 8 && j < NV; ++j) fr[j] = frag[64 * (NK + j)];
    f32x4 kg[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) kg[b] = *reinterpret_cast<const f32x4*>(raw + Y::KG + 4 * (8 * b + 4 * hh));
    __builtin_amdgcn_sched_barrier(0);
    // element i of x: token 8 (i / 4) + 4 hh + i % 4
#pragma unroll
    for (int i2 = 0; i2 < 16; ++i2) x[i2] *= kg[i2 >> 2][i2 & 3];
    auto sees = [&](int i2) {
      const int t = tile * TILE + 8 * (i2 >> 2) + 4 * hh + (i2 & 3);
      return (t <= ((valid >> (i2 >> 3)) & 1 ? pos : -1)) & (t > lo);
    };
    const bool masked = (tile < all0) | (tile >= all1) | (valid != 3);
    if (__builtin_expect(!whole_now, 0) && masked) {
#pragma unroll
      for (int i2 = 0; i2 < 16; ++i2) x[i2] = sees(i2) ? x[i2] : NEG_INF;
    }
    float mx = x[0];
#pragma unroll
    for (int i2 = 1; i2 < 16; ++i2) mx = fmaxf(mx, x[i2]);
    if (__any(mx > limit)) {
      const uint32_t bits = __float_as_uint(mx);
      const auto sw = __builtin_amdgcn_permlane32_swap(bits, bits, false, false);
      const float top = max2(m, max2(__uint_as_float(sw[0]), __uint_as_float(sw[1])));
      const float mu_new = base_less(top, cs);
      const float alpha = __builtin_amdgcn_exp2f(__builtin_fmaf(m, cs, mu_new - BASE));
      m = top;
      mu = mu_new;
      limit = top == NEG_INF ? NEG_INF : top + HEADROOM / cs;
      l *= alpha;
#pragma unroll
      for (int d = 0; d < DT; ++d) acc[d] *= alpha;
    }
    f16x8 wf[2];
#pragma unroll
    for (int i2 = 0; i2 < 16; i2 += 2) {
      const mxq_f32x2 pair = {__builtin_amdgcn_exp2f(__builtin_fmaf(x[i2], cs, mu)),
                              __builtin_amdgcn_exp2f(__builtin_fmaf(x[i2 + 1], cs, mu))};
      l += pair.x + pair.y;                    // of this lane half's tokens
      const f16x2 hp = __builtin_convertvector(pair, f16x2);
      wf[i2 >> 3][i2 & 7] = hp.x;
      wf[i2 >> 3][(i2 & 7) + 1] = hp.y;
    }
    // The weights of a border tile, and those of columns with a bump.  (Out of line,
    // and without a second copy of the products: with one the compiler moves the
    // sums about, 968 us for the prompt chunks against 793.)
    if (__builtin_expect(!whole_now | apart, 0)) {
      f32x4 f[4];
      if (is_whole(tile, valid)) {
#pragma unroll
        for (int b = 0; b < 4; ++b) f[b] = f32x4{1, 1, 1, 1} * __builtin_ldexpf(1.0f, -bump);
      } else {
#pragma unroll
        for (int b = 0; b < 4; ++b) f[b] = *reinterpret_cast<const f32x4*>(raw + Y::VG + 4 * (8 * b + 4 * hh));
        if (masked) {
#pragma unroll
          for (int i2 = 0; i2 < 16; ++i2) f[i2 >> 2][i2 & 3] = sees(i2) ? f[i2 >> 2][i2 & 3] : 0.0f;
        }
        float smax = 0.0f;
#pragma unroll
        for (int i2 = 0; i2 < 16; ++i2) smax = fmaxf(smax, f[i2 >> 2][i2 & 3]);
        const uint32_t bits = __float_as_uint(smax);
        const auto sw = __builtin_amdgcn_permlane32_swap(bits, bits, false, false);
        const int e = max(bump, (int)(max(sw[0], sw[1]) >> 23) - 126 - e_ref);
        if (__any(e > bump)) {
          const float grow = __builtin_ldexpf(1.0f, bump - e);
          bump = e;
          bumped = true;
#pragma unroll
          for (int d = 0; d < DT; ++d) acc[d] *= grow;
        }
#pragma unroll
        for (int i2 = 0; i2 < 16; ++i2) f[i2 >> 2][i2 & 3] = __builtin_ldexpf(f[i2 >> 2][i2 & 3], -(e_ref + bump));
      }
#pragma unroll
      for (int i2 = 0; i2 < 16; i2 += 2) {
        const mxq_f32x2 pair = {(float)wf[i2 >> 3][i2 & 7] * f[i2 >> 2][i2 & 3],
                                (float)wf[i2 >> 3][(i2 & 7) + 1] * f[i2 >> 2][(i2 & 3) + 1]};
        const f16x2 hp = __builtin_convertvector(pair, f16x2);
        wf[i2 >> 3][i2 & 7] = hp.x;
        wf[i2 >> 3][(i2 & 7) + 1] = hp.y;
      }
    }
#pragma unroll
    for (int v0 = 0; v0 < NV; v0 += 8) {
      if (v0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) fr[j] = frag[64 * (NK + v0 + j)];
      }
#pragma unroll
      for (int j = 0; j < 8 && j < NV; ++j)
        acc[(v0 + j) % DT] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, fr[j]),
                                                                    wf[(v0 + j) / DT], acc[(v0 + j) % DT], 0, 0, 0);
    }
  };

  if (count > 0) {
    const int phases = (count + PH - 1) / PH;
    const bool late = wave >= W / 2;
    loads_barrier<2 * PH * Y::JW>();           // phase 0 is here
    scale_of(0, 0);
    for (int i = 0; i < PH; ++i) fill(0, i, 0);
    loads_barrier<PH * Y::JW>();               // its fragments, and phase 1
    for (int p = 0; p < phases; ++p) {
      issue(p + 3, 3);
      // V' of this phase may be on a larger Sref than the sums
      if (e_fill > e_ref) {
        const int up = e_fill - e_ref, take = min(bump, up);
        const float grow = __builtin_ldexpf(1.0f, take - up);
        e_ref = e_fill;
        bump -= take;
#pragma unroll
        for (int d = 0; d < DT; ++d) acc[d] *= grow;
      }
      // Whole tiles take sums on the shared Sref.  A bump up to 64 is undone: the sums
      // stay below 2^15 2^16 2^30 2^64 (weight, V', tokens).  Columns with a larger one
      // stay apart, and weigh by it.
      if (__builtin_expect(bumped, 0)) {
        const int tile = tiles.x + p * PH;
        apart = (tile + PH > w0) & (tile < w1);
        if (apart) {
          const int back = bump <= 64 ? bump : 0;
          const float grow = __builtin_ldexpf(1.0f, back);
          bump -= back;
          apart = bumped = __any(bump > 0);
#pragma unroll
          for (int d = 0; d < DT; ++d) acc[d] *= grow;
        }
      }
      whole_now = whole_next;
      scale_of(p + 1, 1);
#pragma unroll 1
      for (int k = 0; k < 2 * PH; ++k) {
        if (((k & 1) != 0) == late) attend(p, k >> 1);
        else fill(p + 1, k >> 1, 1);           // behind the last phase: page 0, unused
      }
      ok >>= 2 * PH;
      loads_barrier<PH * Y::JW>();             // the fragments of p + 1, and phase p + 2
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");              // no load may write LDS after the workgroup has ended
  {
    const uint32_t bits = __float_as_uint(l);
    const auto sw = __builtin_amdgcn_permlane32_swap(bits, bits, false, false);
    l = __uint_as_float(sw[0]) + __uint_as_float(sw[1]);
  }
  const float f = l == 0.0f ? 0.0f : __builtin_ldexpf(1.0f / l, e_ref + bump - 4);
  store_index(a, u, h);
  if (!have) return;
  const int64_t pr = ((int64_t)uid * cc.H + h) * Y::CT + wave * 32 + c;
  if (hh == 0) store_lse(a, u, pr, row, m * cs, l);
  // the lane holds the values DT r + d of its column, r = 8 (i / 4) + 4 hh + i % 4
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float v[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) v[d] = acc[d][i] * f;
    store_run<D, DT>(a, u, pr, row, DT * (8 * (i >> 2) + 4 * hh + (i & 3)), v);
  }
}

// Joins the chunks of one (token, head): weights 2^(lse_s - lse).  Every chunk
// has written its row, an empty one zeros; a NaN in a chunk's sum or row reaches
// the output.  RW waves
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
  RequestRows own;
  const int64_t b = request_of(a.c, tq, a.T, own);
  if (b < 0) return;                           // a row of no request is left as it was
  const int2 ix = a.part_index[b];
  const int chunks = ix.y;
  if (chunks <= 1) return;                     // written by its only chunk
  const int h = (int)(head / a.G);
  const int64_t j = (tq - own.begin) * a.G + (head - (int64_t)h * a.G);
  const int64_t stride = (int64_t)a.c.H * CT;  // of a chunk
  const int64_t unit = ix.x + j / CT * chunks;  // of chunk 0
  if (unit < 0 || unit + chunks > a.units) return;   // offsets out of order name more units than the grid has
  const int64_t first = (unit * a.c.H + h) * CT + j % CT;
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
        for (int q = 0; q < DL; ++q) o[q] += k + i * RW < n ? wk[i] * v[i][q] : 0.0f;
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
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  uint16_t* out = a.out + tq * a.o_token + head * a.o_head + lane * DL;
#pragma unroll
  for (int q = 0; q < DL; ++q) out[q] = (uint16_t)f32x2_to_bf16x2(o[q] * inv, 0.0f);
  if (a.lse && lane == 0)
    a.lse[row] = total == 0.0f ? NEG_INF : (mx + __builtin_amdgcn_logf(total)) * 0.693147180559945309f;
}

template <int D, int NQ>
static hipError_t launch_few(const AttnArgs& a, dim3 grid, hipStream_t st) {
  static std::atomic<uint32_t> done{0};
  hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(&attention_few_kernel<D, NQ>), few_lds<D, NQ>(), done);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attention_few_kernel<D, NQ>), grid, dim3(64 * FEW_WAVES), (few_lds<D, NQ>()), st, a);
  return hipGetLastError();
}

template <int D>
static hipError_t launch_attention_d(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  const dim3 grid((unsigned)(a.c.H * p.units));
  if (p.waves) {
    constexpr int lds = ManyLayout<D>::LDS;
    static std::atomic<uint32_t> done{0};
    hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(&attention_many_kernel<D>), lds, done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(attention_many_kernel<D>, grid, dim3(64 * MANY_WAVES), lds, st, a);
  } else {
    hipError_t e = hipSuccess;
    if (p.nq == 1) e = launch_few<D, 1>(a, grid, st);
    else if constexpr (D <= 128) e = launch_few<D, 2>(a, grid, st);
    if (e != hipSuccess) return e;
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
