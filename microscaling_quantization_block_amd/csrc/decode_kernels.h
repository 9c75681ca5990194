// Host-side launchers of the few-row products and of the 4-bit cache
// (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq.h"

namespace mxq {

struct GemvArgs {
  const uint16_t* x;
  int64_t ld_x, x_rows;
  const uint8_t* w;             // packed codes, group g at w + g * w_group
  int64_t ld_w, w_group;        // bytes
  const uint8_t* scales;        // group g at scales + g * s_group
  int64_t s_group;
  const float* gs;              // one per group
  int64_t M, N, K;              // N: output columns (SwiGLU: the weight has 2 N rows)
  uint16_t* y;
  int64_t ld_y;
  int num_groups;               // 0: dense
  const int32_t* offsets;
  const int32_t* row_index;
};
enum GemvScales { GS_ROW = 0, GS_MFMA = 1, GS_TILE = 2 };
hipError_t launch_nvfp4_gemv(const GemvArgs& a, GemvScales layout, bool swiglu, hipStream_t st);

// The pages of an NVFP4 cache (mxq_cache), by value.
struct CacheArgs {
  uint8_t *kc, *ks, *vc, *vs;   // codes, block scales
  float *kg, *vg;               // second scales
  int64_t pages, pc, psc, pg;   // page strides: code bytes, scale bytes, second scales
  int H, D, P_log2;
  const int32_t* table;         // [B, width], ld entries a row
  int64_t ld_table, width;
  const int32_t* seq_lens;
  const int32_t* q_offsets;     // [B + 1], or nullptr: one token per request
  int64_t B;
};

struct AppendArgs {
  CacheArgs c;
  const uint16_t *k, *v;
  int64_t T, k_token, k_head, v_token, v_head;    // strides, elements
  uint16_t *k_dq, *v_dq;        // [T, H, D], or nullptr
};
hipError_t launch_cache_append(const AppendArgs& a, hipStream_t st);

struct AttnArgs {
  CacheArgs c;
  const uint16_t* q;
  int64_t T, q_token, q_head;   // strides, elements
  int Hq, G;                    // G = Hq / H query heads share a KV head
  float scale_log2;             // scale * log2(e)
  int64_t window;               // 0: none
  uint16_t* out;
  int64_t o_token, o_head;
  float* lse;                   // [T, Hq], or nullptr
  // partial results (target > 0): of unit i, KV head h and column j of its tile the
  // normalized row and its log2 sum at (i H + h) CT + j, and of each request its first
  // unit and its chunks
  float *part_o, *part_lse;
  int2* part_index;
  // chunks of all requests: at most `target` beside one per column tile, `coarse` if that
  // makes none longer than LONG_CHUNK; target 0: a request's context is one chunk
  int target, coarse;
  int64_t units;                // of the grid (times the KV heads)
};

constexpr int MANY_WAVES = 8;                  // waves of a workgroup with many columns
constexpr int MIN_CHUNK = 8;                   // 32-token tiles of the shortest chunk
// Two workgroups per compute unit as long as a chunk stays below 2048 tokens,
// else six: 64 contexts up to 4096 took 53.8, 56.4, 57.7 us with 512, 768, 1536
// workgroups aimed at, four contexts up to 131071 110, 104, 93.5.
constexpr int LONG_CHUNK = 64;
// No split, and no second launch, where unsplit contexts of at most 2048 tokens
// give every compute unit a workgroup: 32 contexts up to 1000 tokens, 8 heads
// 15.6 us, split 19.1; 64 up to 2048 32.1 and 35.3.  From 128 workgroups on: 24
// up to 2048 (192 workgroups) 24.1 and 21.6.
constexpr int ENOUGH = 256;

// How a call is cut (no row sees more than max_context tokens): column tiles
// of ct (query, head) pairs, and the number of work units (a bound).
struct AttnPlan {
  int nq, waves, ct, target, coarse;
  int64_t units;
};
inline AttnPlan plan_attention(int64_t B, int64_t T, int H, int G, int D, int64_t max_context, bool ragged) {
  AttnPlan p;
  // columns of an average request: a few fit one or two tiles of a wave, and
  // the waves of a workgroup share the context; many are spread over the waves
  const int64_t cols = (T + B - 1) / B * G;
  const int nq_max = D <= 128 ? 2 : 1;
  p.waves = cols > 16 * nq_max ? MANY_WAVES : 0;
  p.nq = cols > 16 ? 2 : 1;
  p.ct = p.waves ? 32 * p.waves : 16 * p.nq;
  const int64_t tiles = ragged ? T * G / p.ct + B : B * ((G + p.ct - 1) / p.ct);
  // workgroups aimed at
  const int64_t want = p.waves ? 256 : 1536, few = p.waves ? 256 : 512;
  const int64_t most = (max_context + 32 * MIN_CHUNK - 1) / (32 * MIN_CHUNK);   // chunks of the longest context
  const bool enough = !p.waves && tiles * H >= ENOUGH && max_context <= 32 * LONG_CHUNK;
  p.target = most <= 2 || enough || tiles * H >= 4 * want ? 0 : (int)((want + H - 1) / H);
  p.coarse = (int)((few + H - 1) / H);
  const int64_t bound = tiles * most;
  p.units = p.target ? (tiles + p.target < bound ? tiles + p.target : bound) : tiles;
  return p;
}
inline int64_t attention_workspace(const AttnPlan& p, int64_t B, int H, int D) {
  return p.target ? p.units * H * p.ct * (D + 1) * (int64_t)sizeof(float) + B * (int64_t)sizeof(int2) : 0;
}
hipError_t launch_attention(const AttnArgs& a, const AttnPlan& p, hipStream_t st);

}  // namespace mxq
