// Rotary positions for a call's queries and keys, keys and values quantized into
// the pages of an NVFP4 cache on the way.
//
// The pair i of a row at position p turns by p inv_freq[i]; its cosine and sine
// are taken in binary64 (a far position's angle has no digits left in
// binary32) and rounded to binary32, the products and their sum are one
// rounding each, and the turned row is rounded to BF16 before it is quantized: the
// cache gets the bytes that nvfp4_cache_append writes for the turned rows.
//
// A wave holds one token, or a share of its heads: it finds the token's request,
// position and page once, a lane computes one angle, and the lanes then keep the eight
// cosines and sines of their place in a row for all heads.  D / 8 lanes hold a row;
// a half layout's partner values come from another lane of the row.  Prompts are bound by
// memory: 9.7 k tokens of 32 + 16 heads of 128, 250 MB in 49.1 us, 5.1 TB/s; a decode
// step by one chain of latencies: 128 tokens 4.5 us (a launch alone is about 2).  The heads
// are loaded before the token's request and page are looked up; behind the look-ups, and
// with the source of a row chosen among kernel arguments, prompts took 60 us.

#include "cache_device.h"
#include "layer_kernels.h"

namespace mxq {

namespace {

// Cosine and sine of x in binary64, |x| below 2^40 or so.  x - n pi/2 in two
// steps: n times the first part of pi/2 is a multiple of 2^-52, and so is what
// is left of x, below 2, which is therefore exact; the second part's
// product is then far smaller.  Taylor series on [-pi/4, pi/4]: what is left out is
// below 2^-58.
__device__ __forceinline__ void cos_sin(double x, double& c, double& s) {
  const double n = __builtin_rint(x * 0.63661977236758134308);          // 2 / pi
  double r = __builtin_fma(-n, 1.57079632679489655800, x);
  r = __builtin_fma(-n, 6.12323399573676603587e-17, r);
  const double z = r * r;
  double a = 1.0 / 355687428096000.0;                                    // 1 / 17!
  a = __builtin_fma(a, z, -1.0 / 1307674368000.0);
  a = __builtin_fma(a, z, 1.0 / 6227020800.0);
  a = __builtin_fma(a, z, -1.0 / 39916800.0);
  a = __builtin_fma(a, z, 1.0 / 362880.0);
  a = __builtin_fma(a, z, -1.0 / 5040.0);
  a = __builtin_fma(a, z, 1.0 / 120.0);
  a = __builtin_fma(a, z, -1.0 / 6.0);
  const double sr = __builtin_fma(r * z, a, r);
  double b = -1.0 / 6402373705728000.0;                                  // -1 / 18!
  b = __builtin_fma(b, z, 1.0 / 20922789888000.0);
  b = __builtin_fma(b, z, -1.0 / 87178291200.0);
  b = __builtin_fma(b, z, 1.0 / 479001600.0);
  b = __builtin_fma(b, z, -1.0 / 3628800.0);
  b = __builtin_fma(b, z, 1.0 / 40320.0);
  b = __builtin_fma(b, z, -1.0 / 720.0);
  b = __builtin_fma(b, z, 1.0 / 24.0);
  b = __builtin_fma(b, z, -0.5);
  const double cr = __builtin_fma(b, z, 1.0);
  const int q = (int)((int64_t)n & 3);
  const double cc = q & 1 ? sr : cr, ss = q & 1 ? cr : sr;
  c = q == 1 || q == 2 ? -cc : cc;
  s = q & 2 ? -ss : ss;
}

constexpr int BATCH = 4;                       // rows of a lane in flight

template <int D, bool INTERLEAVED>
__global__ __launch_bounds__(256) void rope_append_kernel(RopeArgs a) {
  constexpr int L = D / 8, ROWS = 64 / L;      // lanes of a row, rows of a wave
  constexpr int PAIRS = INTERLEAVED ? 4 : 8;   // of a lane
  __shared__ float2 turns[4][D / 2];
  const CacheArgs& c = a.p.c;
  // the wave's number in a scalar register, so that what it looks up by its token
  // are scalar loads, which wait for no vector load
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), in_wave = threadIdx.x & 63, lane = in_wave & (L - 1);
  const uint32_t unit = blockIdx.x * 4 + wave, token = unit / (uint32_t)a.split;
  const int64_t t = token;
  if (t >= a.p.T) return;                      // whole waves
  constexpr int ANGLES = (D / 2 + 63) / 64;    // of a lane
  float freq[ANGLES];
#pragma unroll
  for (int i = 0; i < ANGLES; ++i) freq[i] = a.inv_freq[min(in_wave + 64 * i, a.rot / 2 - 1)];

  // the token's heads: q, k, v in turn; this wave's share of them
  const int heads = a.Hq + 2 * c.H, passes = (heads + ROWS - 1) / ROWS;
  const int share = (int)(unit - token * (uint32_t)a.split);
  const int first = passes * share / a.split, last = passes * (share + 1) / a.split;
  const int own = in_wave / L;
  // where the token's k and v lie from its q, and the strides of the heads, as plain
  // numbers in scalar registers: a choice between kernel arguments would be loaded, row by row
  const uint16_t* q = a.q + t * a.q_token;
  int64_t to_k = (a.p.k + t * a.p.k_token) - q, to_v = (a.p.v + t * a.p.v_token) - q;
  int64_t q_head = a.q_head, k_head = a.p.k_head, v_head = a.p.v_head;
  asm("" : "+s"(to_k), "+s"(to_v), "+s"(q_head), "+s"(k_head), "+s"(v_head));
  const auto load = [&](int p0, uint4* x) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int h = (p0 + i) * ROWS + own, kv = h - a.Hq;
      const bool is_q = kv < 0, is_k = kv < c.H;
      const uint16_t* head = q + (is_q ? h * q_head : is_k ? to_k + kv * k_head : to_v + (kv - c.H) * v_head);
      x[i] = p0 + i < last && h < heads ? load16_once(head + 8 * lane) : make_uint4(0, 0, 0, 0);
    }
  };
  // on their way while the request, the page and the angles are found
  uint4 x[BATCH];
  load(first, x);

  RequestRows rows;
  const int64_t b = request_of(c, t, a.p.T, rows);
  if (b < 0) return;
  const int64_t pos = (int64_t)c.seq_lens[b] - rows.len + (t - rows.begin);
  const int64_t page = page_of(c, b, pos);

  float2* turn = turns[wave];
#pragma unroll
  for (int i = 0; i < ANGLES; ++i) {
    double co, si;
    cos_sin((double)pos * (double)freq[i], co, si);
    if (in_wave + 64 * i < a.rot / 2) turn[in_wave + 64 * i] = make_float2((float)(co * a.factor), (float)(si * a.factor));
  }
  // the wave's own writes, before any of its lanes reads them
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  const bool turned = 8 * lane < a.rot;
  const int half = a.rot / 16;                 // lanes of half the turned values
  const bool second = !INTERLEAVED && lane >= half;
  float co[PAIRS], si[PAIRS];
  if (turned) {
    const float2* at = turn + (INTERLEAVED ? 4 * lane : 8 * (second ? lane - half : lane));
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
      const float2 v = at[i];
      co[i] = v.x;
      si[i] = second ? v.y : -v.y;             // the partner's factor
    }
  }
  const int partner = in_wave - lane + (second ? lane - half : lane + half);

  for (int p0 = first; p0 < last; p0 += BATCH) {
    if (p0 > first) load(p0, x);
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int h = (p0 + i) * ROWS + own;
      if (p0 + i >= last) break;               // the same for the whole wave
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t o[4];
      if constexpr (INTERLEAVED) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // (u, v) -> (u c - v s, v c + u s); si holds -s
          const float u = bf16_lo(w[j]), v = bf16_hi(w[j]);
          o[j] = f32x2_to_bf16x2(u * co[j] + v * si[j], v * co[j] - u * si[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t y = (uint32_t)__shfl((int)w[j], partner, 64);
          o[j] = f32x2_to_bf16x2(bf16_lo(w[j]) * co[2 * j] + bf16_lo(y) * si[2 * j],
                                 bf16_hi(w[j]) * co[2 * j + 1] + bf16_hi(y) * si[2 * j + 1]);
        }
      }
      if (h >= heads) continue;                // whole rows: the lane exchanges below stay inside a row
      const bool is_v = h >= a.Hq + c.H;
      const uint4 y = turned && !is_v ? make_uint4(o[0], o[1], o[2], o[3]) : x[i];
      if (h < a.Hq) {
        store16_once(a.q_out + t * a.o_token + h * a.o_head + 8 * lane, y);
      } else {
        const int kv = is_v ? h - a.Hq - c.H : h - a.Hq;
        uint16_t* dq = is_v ? a.p.v_dq : a.p.k_dq;
        append_row<D>(c, is_v, kv, page, pos, lane, y, dq ? dq + (t * c.H + kv) * D : nullptr);
      }
    }
  }
}

template <int D>
void launch_rope(const RopeArgs& a, dim3 grid, hipStream_t st) {
  if (a.interleaved) hipLaunchKernelGGL((rope_append_kernel<D, true>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((rope_append_kernel<D, false>), grid, dim3(256), 0, st, a);
}

}  // namespace

hipError_t launch_rope_append(const RopeArgs& args, hipStream_t st) {
  RopeArgs a = args;
  const int D = a.p.c.D, rows = 512 / D, passes = (a.Hq + 2 * a.p.c.H + rows - 1) / rows;
  // four waves for every SIMD where there are tokens enough; else a token's heads are shared out
  const int64_t want = 4096 / a.p.T;
  a.split = (int)(want < 1 ? 1 : want < passes ? want : passes);
  const dim3 grid((unsigned)((a.p.T * a.split + 3) / 4));
  if (D == 64) launch_rope<64>(a, grid, st);
  else if (D == 128) launch_rope<128>(a, grid, st);
  else launch_rope<256>(a, grid, st);
  return hipGetLastError();
}

}  // namespace mxq
