// The router of a layer with experts, the rows of its tokens ordered by expert,
// and the way there and back with its gradients.
//
// Router: a token's k largest logits, ties to the lower expert, and their softmax weights
// (over the chosen ones, or over all experts).  A token is 16 lanes or a wave, expert
// v LANES + lane in lane.  Bound by its instructions and their latency: every
// lane sorts its few logits once, and a round compares the lanes' first ones.  64
// tokens of 128 experts, top 8: 7.1 us with their rows; 8192 tokens: 5.6 us, the rows 6.0, the
// gradient of the logits 5.0 (the largest key searched anew in each round: 10.7 us).
//
// Order: rows by (expert, token, slot), a counting sort.  Each group of tokens
// counts its slots by expert; a second kernel adds the counts of the groups before its own
// and of the experts before each, and gives every slot its row: lanes with the same
// expert rank themselves by ballots over the bits of the expert's number, so that no
// order depends on the timing of atomics.  Few tokens are routed and sorted by one workgroup in one launch.
//
// There and back: a lane owns eight columns; all of a token's rows are in flight
// at once, so these are copies bound by memory.  8192 tokens of 2048 values, eight rows
// each: to the rows 49 us (302 MB), back 51, the gradient of the way back 76 (436 MB). The
// experts' rows, far more than a cache holds, go past the caches (to and back 135 us
// together where they do not); tokens' rows, which the next step reads, do not.

#include "lanes.h"
#include "layer_kernels.h"

namespace mxq {

namespace {

// A logit and its expert as one unsigned integer: larger logits are larger, and
// of equal ones that of the lower expert.  The upper half orders values: both
// zeros give one number, a NaN the largest.  0 stands for an expert that is not
// there (any more).  Binary32 logits take 64 bits, BF16 ones 32.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t order) {
  return __uint_as_float(order & 0x80000000u ? order & 0x7FFFFFFFu : ~order);      // 0xFFFFFFFF: a NaN
}
constexpr uint32_t ORDER_MINUS_INF = 0x007FFFFFu;

template <bool F32>
struct Key;
template <>
struct Key<true> {
  using T = uint64_t;
  static __device__ __forceinline__ T make(float x, int e) { return (uint64_t)order_of(x) << 32 | (uint32_t)~e; }
  static __device__ __forceinline__ bool chosen(T k) { return (uint32_t)(k >> 32) > ORDER_MINUS_INF; }
  static __device__ __forceinline__ float value(T k) { return value_of((uint32_t)(k >> 32)); }
  static __device__ __forceinline__ int expert(T k) { return (int)~(uint32_t)k; }
  template <int LANES>
  static __device__ __forceinline__ T largest(T k) {
    const uint32_t hi = lanes_max<LANES>((uint32_t)(k >> 32));
    const uint32_t lo = lanes_max<LANES>((uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return (uint64_t)hi << 32 | lo;
  }
};
template <>
struct Key<false> {
  using T = uint32_t;
  static __device__ __forceinline__ T make(float x, int e) { return (order_of(x) & 0xFFFF0000u) | (0xFFFFu - e); }
  static __device__ __forceinline__ bool chosen(T k) { return k >> 16 > ORDER_MINUS_INF >> 16; }
  static __device__ __forceinline__ float value(T k) { return value_of(k & 0x80000000u ? k & 0xFFFF0000u : k | 0xFFFFu); }
  static __device__ __forceinline__ int expert(T k) { return 0xFFFF - (int)(k & 0xFFFFu); }
  template <int LANES>
  static __device__ __forceinline__ T largest(T k) { return lanes_max<LANES>(k); }
};

// Sorts a[0 .. N - 1], the largest first: Batcher's odd-even merge sort, all
// places known at compile time.
template <int N, class T>
__device__ __forceinline__ void sort_down(T* a) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const T x = a[i + j], y = a[i + j + k];
            a[i + j] = x > y ? x : y;
            a[i + j + k] = x > y ? y : x;
          }
}

template <bool F32>
__device__ __forceinline__ float logit(const void* logits, int64_t i) {
  if constexpr (F32) return static_cast<const float*>(logits)[i];
  return __uint_as_float((uint32_t)static_cast<const uint16_t*>(logits)[i] << 16);
}

// The logits of this lane, all loads in flight at once: a lane beyond the last
// expert reads that one (a load in a branch of its own would be waited for there).
template <int LANES, int VPL, bool F32>
__device__ __forceinline__ void load_logits(const void* logits, int64_t at, int E, int lane, float* x) {
#pragma unroll
  for (int v = 0; v < VPL; ++v) x[v] = logit<F32>(logits, at + min(v * LANES + lane, E - 1));
}

constexpr int SORT_WAVES = 8;

// Routes token t (LANES lanes, `lane` of them); `count` gets every slot and its expert
// (-1: none).  A lane sorts its own keys once; a round then compares the lanes'
// first ones and the lane that has the largest drops it.
template <int LANES, int VPL, bool F32, class F>
__device__ __forceinline__ void route_token(const MoeArgs& a, int64_t t, int lane, F&& count) {
  using K = Key<F32>;
  float x[VPL];
  load_logits<LANES, VPL, F32>(a.logits, t * a.ld, a.E, lane, x);
  typename K::T key[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int e = v * LANES + lane;
    const typename K::T k = K::make(x[v], e);
    key[v] = e < a.E ? k : 0;
  }
  sort_down<VPL>(key);
  typename K::T top = K::template largest<LANES>(key[0]);
  const float largest = K::value(top);
  float all = 0.0f;
  if (!a.renorm) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const float p = expf(x[v] - largest);
      all += v * LANES + lane < a.E ? p : 0.0f;
    }
    all = lanes_sum<LANES>(all);
  }
  typename K::T mine = 0;                      // lane j: the key of slot j
  for (int j = 0; j < a.k; ++j) {
    if (!K::chosen(top)) break;                // nothing is left for this token
    mine = lane == j ? top : mine;
    // bit masks: of a choice between key[v] and key[v + 1] the compiler makes a
    // choice of places, with a chain of comparisons for each
    const typename K::T drop = key[0] == top ? ~(typename K::T)0 : 0;
#pragma unroll
    for (int v = 0; v + 1 < VPL; ++v) key[v] = (key[v + 1] & drop) | (key[v] & ~drop);
    key[VPL - 1] &= ~drop;
    top = K::template largest<LANES>(key[0]);
  }
  const bool has = mine != 0;
  const int e = has ? K::expert(mine) : -1;
  const float part = has ? expf(K::value(mine) - largest) : 0.0f;
  const float total = a.renorm ? lanes_sum<LANES>(part) : all;
  if (lane < a.k) {
    a.experts[t * a.k + lane] = e;
    a.weights[t * a.k + lane] = has ? part / total : 0.0f;
    count(t * a.k + lane, e);
  }
}

// Inclusive sum over the lanes of a wave: shifts inside 16 lanes, then the last
// lanes of 16 and of 32 to those behind them.
__device__ __forceinline__ int wave_running_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
  return v + __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
}

// The sum of n over the workgroup's threads before this one.  `scratch` holds an int per wave.
template <int THREADS>
__device__ __forceinline__ int block_exclusive_sum(int n, int* scratch) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int s = wave_running_sum(n);
  if (lane == 63) scratch[wave] = s;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 64; ++i) before += i < wave ? scratch[i] : 0;
  return before + s - n;
}

// LDS of the sort: two counts of every expert (of all groups, and of those before
// this workgroup's) as one 64-bit number, then hist [SORT_WAVES, E].
inline size_t sort_lds(int E) { return (size_t)E * 8 + (size_t)SORT_WAVES * E * 4; }

__device__ __forceinline__ int pieces_of_wave(int slots) { return ((slots + 63) / 64 + SORT_WAVES - 1) / SORT_WAVES; }
__device__ __forceinline__ int* sort_hist(int* lds, int E) { return lds + 2 * E; }

// Gives the slots [first, last) of the call (this workgroup's) their rows; `ids`
// holds their experts, ids[0] that of slot `first`.
// GROUPS: their counts and those of the other groups are in a.counts; else they are all there is.
// COUNTED: they are counted in hist, slot s in wave s / (64 pieces_of_wave).
template <int THREADS, bool GROUPS, bool COUNTED>
__device__ __forceinline__ void sort_slots(const MoeArgs& a, int64_t group, int64_t first, int64_t last, const int* ids,
                                           int* lds) {
  __shared__ int scratch[THREADS / 64];
  __shared__ int all_rows;
  const int E = a.E, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, slots = (int)(last - first);
  uint64_t* both = reinterpret_cast<uint64_t*>(lds);           // of all groups << 32 | of the groups before
  int* hist = sort_hist(lds, E);

  // a lane adds eight experts' counts over every slices-th group; the first eight
  // of them are on their way while the workgroup's own slots are counted.  Not more
  // slices than make 256 groups eight each: few experts would have many lanes add
  // to the same place (8 experts, 8192 tokens: 10.0 us with 512 slices)
  const int per_row = (E + 7) / 8, slices = min(THREADS / per_row, 32);
  const int col = threadIdx.x % per_row, slice = threadIdx.x / per_row;
  constexpr int AHEAD = 8;
  uint4 ahead[AHEAD];
  if constexpr (GROUPS) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int64_t g = min(slice + (int64_t)i * slices, a.groups - 1);
      ahead[i] = *reinterpret_cast<const uint4*>(a.counts + (g * per_row + col) * 8);
    }
  }
  if constexpr (!COUNTED)
    for (int i = threadIdx.x; i < (SORT_WAVES + 2) * E; i += THREADS) lds[i] = 0;
  // whole 64-slot pieces of the workgroup's slots, in order, to the waves in order
  const int each = pieces_of_wave(slots), from = wave * each * 64;
  const int to = min(slots, from + each * 64);
  const auto expert_at = [&](int s) {          // E stands for no expert
    const int e = s < to ? ids[s] : -1;
    return (unsigned)e < (unsigned)E ? e : E;
  };
  const int first_e = wave < SORT_WAVES ? expert_at(from + lane) : E;
  if constexpr (!COUNTED) {
    __syncthreads();
    if (wave < SORT_WAVES)
      for (int s0 = from; s0 < to; s0 += 64) {
        const int e = s0 == from ? first_e : expert_at(s0 + lane);
        if (e < E) atomicAdd(&hist[wave * E + e], 1);
      }
  }
  if constexpr (GROUPS) {
    uint32_t sum[8], pre[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = pre[i] = 0;
    const auto add = [&](uint4 w, int64_t g) {
      const uint32_t n[4] = {w.x, w.y, w.z, w.w};
      const uint32_t in = g < a.groups ? 0xFFFFFFFFu : 0u, earlier = g < group ? 0xFFFFFFFFu : 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = n[i] & 0xFFFFu, hi = n[i] >> 16;
        sum[2 * i] += lo & in;
        sum[2 * i + 1] += hi & in;
        pre[2 * i] += lo & earlier;
        pre[2 * i + 1] += hi & earlier;
      }
    };
    if (slice < min((int64_t)slices, a.groups)) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) add(ahead[i], slice + (int64_t)i * slices);
#pragma unroll 4
      for (int64_t g = slice + (int64_t)AHEAD * slices; g < a.groups; g += slices)
        add(*reinterpret_cast<const uint4*>(a.counts + (g * per_row + col) * 8), g);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col * 8 + i < E)
          atomicAdd(reinterpret_cast<unsigned long long*>(&both[col * 8 + i]), (unsigned long long)sum[i] << 32 | pre[i]);
    }
  }
  if constexpr (!COUNTED) __syncthreads();
  // the experts' first rows, then those of this workgroup's waves
  const auto total = [&](int e) {
    if constexpr (GROUPS) return (int)(both[e] >> 32);
    int n = 0;
#pragma unroll
    for (int w = 0; w < SORT_WAVES; ++w) n += hist[w * E + e];
    return n;
  };
  const int per = (E + THREADS - 1) / THREADS, e0 = min(E, (int)threadIdx.x * per), e1 = min(E, e0 + per);
  int n = 0;
  for (int e = e0; e < e1; ++e) n += total(e);
  int start = block_exclusive_sum<THREADS>(n, scratch);
  for (int e = e0; e < e1; ++e) {
    if (group == 0) a.offsets[e] = start;
    int at = start + (GROUPS ? (int)(uint32_t)both[e] : 0);
    start += total(e);
#pragma unroll
    for (int w = 0; w < SORT_WAVES; ++w) {
      const int m = hist[w * E + e];
      hist[w * E + e] = at;
      at += m;
    }
  }
  if (threadIdx.x == THREADS - 1) {            // the last thread's end is the sum of all
    if (group == 0) a.offsets[E] = start;
    all_rows = start;
  }
  __syncthreads();
  const int64_t rows = all_rows;
  const int bits = 32 - __clz(E);              // of numbers up to E
  if (wave < SORT_WAVES)
    for (int s0 = from; s0 < to; s0 += 64) {
      const int s = s0 + lane;
      const int e = s0 == from ? first_e : expert_at(s);
      uint64_t same = ~0ull;                   // lanes with this expert
      for (int b = 0; b < bits; ++b) {
        const bool one = (e >> b) & 1;
        const uint64_t ones = __ballot(one);
        same &= one ? ones : ~ones;
      }
      const int leader = __ffsll((unsigned long long)same) - 1;
      const int rank = __popcll(same & ((1ull << lane) - 1));
      int at = 0;
      if (lane == leader && e < E) at = atomicAdd(&hist[wave * E + e], __popcll(same));
      at = __shfl(at, leader, 64) + rank;
      // the next piece's counts come after this one's
      __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
      if (s < to) {
        const int64_t slot = first + s;
        a.row_of[slot] = e < E ? at : -1;
        if (e < E) a.row_token[at] = (int)((uint32_t)slot / (uint32_t)a.k);      // slots stay below 2^26
      }
    }
  // rows of no slot: token 0, a row that a gather may read
  for (int64_t r = first + threadIdx.x; r < last; r += THREADS)
    if (r >= rows) a.row_token[r] = 0;
}

// Threads of a workgroup of the router that has `tokens` of `lanes` lanes: one pass
// for 32 tokens of 16 lanes; more fill the workgroup (65536 tokens of 128 experts: 31.8 us
// with 512 threads, 28.2 with 1024, the sort included).
inline int route_threads(int lanes, int64_t tokens) { return lanes * tokens <= 512 ? 512 : 1024; }

template <int LANES, int VPL, bool F32>
__global__ __launch_bounds__(1024) void route_kernel(MoeArgs a) {
  extern __shared__ __align__(16) int lds[];
  const int threads = (int)blockDim.x;
  for (int i = threadIdx.x; i < a.E; i += threads) lds[i] = 0;
  __syncthreads();
  const int64_t first = blockIdx.x * a.group_tokens, last = min(a.T, first + a.group_tokens);
  for (int64_t t = first + threadIdx.x / LANES; t < last; t += threads / LANES)
    route_token<LANES, VPL, F32>(a, t, threadIdx.x & (LANES - 1), [&](int64_t, int e) {
      if (e >= 0) atomicAdd(&lds[e], 1);
    });
  __syncthreads();
  const int pad = (a.E + 7) / 8 * 8;
  for (int i = threadIdx.x; i < pad; i += threads)
    a.counts[blockIdx.x * (int64_t)pad + i] = (uint16_t)(i < a.E ? lds[i] : 0);
}

// Tokens that one workgroup routes in a pass and sorts: their experts stay in LDS.
constexpr int one_tokens(int lanes) { return 1024 / lanes; }

template <int LANES, int VPL, bool F32>
__global__ __launch_bounds__(1024) void route_one_kernel(MoeArgs a) {
  extern __shared__ __align__(16) int lds[];
  __shared__ int ids[one_tokens(LANES) * LANES];         // topk is at most LANES
  int* hist = sort_hist(lds, a.E);
  for (int i = threadIdx.x; i < SORT_WAVES * a.E; i += 1024) hist[i] = 0;
  __syncthreads();
  const int of_wave = 64 * pieces_of_wave((int)a.T * a.k);
  for (int64_t t = threadIdx.x / LANES; t < a.T; t += 1024 / LANES)
    route_token<LANES, VPL, F32>(a, t, threadIdx.x & (LANES - 1), [&](int64_t slot, int e) {
      ids[slot] = e;
      if (e >= 0) atomicAdd(&hist[(int)slot / of_wave * a.E + e], 1);
    });
  __syncthreads();
  sort_slots<1024, false, true>(a, 0, 0, a.T * a.k, ids, lds);
}

__global__ __launch_bounds__(256) void count_kernel(MoeArgs a) {
  extern __shared__ __align__(16) int lds[];
  for (int i = threadIdx.x; i < a.E; i += 256) lds[i] = 0;
  __syncthreads();
  const int64_t first = blockIdx.x * a.group_tokens * a.k, last = min(a.T * a.k, first + a.group_tokens * a.k);
  for (int64_t s = first + threadIdx.x; s < last; s += 256) {
    const int e = a.experts[s];
    if ((unsigned)e < (unsigned)a.E) atomicAdd(&lds[e], 1);
  }
  __syncthreads();
  const int pad = (a.E + 7) / 8 * 8;
  for (int i = threadIdx.x; i < pad; i += 256) a.counts[blockIdx.x * (int64_t)pad + i] = (uint16_t)(i < a.E ? lds[i] : 0);
}

__global__ __launch_bounds__(512) void sort_kernel(MoeArgs a) {
  extern __shared__ __align__(16) int lds[];
  const int64_t slots = a.T * a.k, each = a.group_tokens * a.k, first = blockIdx.x * each;
  sort_slots<512, true, false>(a, blockIdx.x, first, min(slots, first + each), a.experts + first, lds);
}

__global__ __launch_bounds__(1024) void sort_one_kernel(MoeArgs a) {
  extern __shared__ __align__(16) int lds[];
  sort_slots<1024, false, false>(a, 0, 0, a.T * a.k, a.experts, lds);
}

// dl of the softmax: over the chosen experts w_j (dw_j - sum w dw); over all of
// them p_e (dw_e - sum w dw), dw_e 0 where e was not chosen.
template <int LANES, int VPL, bool F32>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteBwdArgs a) {
  const int lane = threadIdx.x & (LANES - 1);
  const int64_t t = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  if (t >= a.T) return;                        // whole groups of LANES lanes leave
  // lane j holds slot j (topk is at most LANES)
  const int64_t slot = t * a.k + min(lane, a.k - 1);
  const int id = a.experts[slot];
  const float w = a.weights[slot], dw = a.dweights[slot];
  const bool has = lane < a.k && id >= 0;
  const float mean = lanes_sum<LANES>(has ? w * dw : 0.0f);
  float d[VPL];
  if (a.renorm) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) d[v] = 0.0f;
  } else {
    float x[VPL], top = -__builtin_inff(), total = 0.0f;
    load_logits<LANES, VPL, F32>(a.logits, t * a.ld, a.E, lane, x);
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      x[v] = v * LANES + lane < a.E ? x[v] : -__builtin_inff();
      top = fmaxf(top, x[v]);
    }
    top = value_of(lanes_max<LANES>(order_of(top)));
    // a token whose experts are all masked has weights of zero: nothing flows
    const float base = top > -__builtin_inff() ? top : 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      x[v] = expf(x[v] - base);
      total += x[v];
    }
    total = lanes_sum<LANES>(total);
    const float r = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) d[v] = -(x[v] * r) * mean;
  }
  const float own = has ? w * (a.renorm ? dw - mean : dw) : 0.0f;
  for (int j = 0; j < a.k; ++j) {
    const int e = __shfl(id, j, LANES);
    const float g = __shfl(own, j, LANES);
#pragma unroll
    for (int v = 0; v < VPL; ++v) d[v] += e == v * LANES + lane ? g : 0.0f;
  }
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int e = v * LANES + lane;
    if (e >= a.E) continue;
    if constexpr (F32) static_cast<float*>(a.dlogits)[t * a.ld_d + e] = d[v];
    else static_cast<uint16_t*>(a.dlogits)[t * a.ld_d + e] = (uint16_t)f32x2_to_bf16x2(d[v], 0.0f);
  }
}

template <int LANES_, int VPL_, bool F32_>
struct Lanes {
  static constexpr int LANES = LANES_, VPL = VPL_;
  static constexpr bool F32 = F32_;
};

// Lanes of a token: 16 up to 128 experts (four tokens a wave), a wave beyond, and where 16 lanes cannot hold the
// choices.  (256 experts, top 8, with 16 lanes of sixteen logits each: 12.2, 14.3 and 18.8 us for 64, 512 and 8192
// tokens; with a wave of four: 9.4, 10.4 and 17.8.)
int lanes_of(int E, int k) { return k <= 16 && E <= 128 ? 16 : 64; }

// Calls f with a Lanes for E experts and k choices.
template <bool F32, class F>
hipError_t with_lanes(int E, int k, F&& f) {
  if (lanes_of(E, k) == 16) {
    if (E <= 16) return f(Lanes<16, 1, F32>());
    if (E <= 64) return f(Lanes<16, 4, F32>());
    return f(Lanes<16, 8, F32>());
  }
  if (E <= 256) return f(Lanes<64, 4, F32>());
  if (E <= 512) return f(Lanes<64, 8, F32>());
  return f(Lanes<64, 16, F32>());
}
template <class F>
hipError_t with_lanes(bool f32, int E, int k, F&& f) {
  return f32 ? with_lanes<true>(E, k, f) : with_lanes<false>(E, k, f);
}

}  // namespace

void plan_moe(MoeArgs& a, bool routed) {
  a.groups = 0;
  a.group_tokens = a.T;
  const int lanes = lanes_of(a.E, a.k);
  // one workgroup routes its pass of tokens, or sorts some slots (512 slots 3.6 us, 4096 9.8, where two launches take 7.1)
  if (routed ? a.T <= one_tokens(lanes) : a.T * a.k <= 2048) return;
  // at least a pass of the router's workgroup; up to 256 groups beyond that, while counts fit 16 bits
  const int64_t pass = lanes == 16 ? 32 : 16;
  int64_t each = (a.T + 255) / 256;
  each = each < pass ? pass : each;
  const int64_t most = 65535 / a.k;
  a.group_tokens = each < most ? each : most;
  a.groups = (a.T + a.group_tokens - 1) / a.group_tokens;
}

hipError_t launch_moe_route(const MoeArgs& a, hipStream_t st) {
  const hipError_t e = with_lanes(a.f32, a.E, a.k, [&](auto lanes) {
    using W = decltype(lanes);
    if (!a.groups)
      hipLaunchKernelGGL((route_one_kernel<W::LANES, W::VPL, W::F32>), dim3(1), dim3(1024), sort_lds(a.E), st, a);
    else
      hipLaunchKernelGGL((route_kernel<W::LANES, W::VPL, W::F32>), dim3((unsigned)a.groups),
                         dim3((unsigned)route_threads(W::LANES, a.group_tokens)), (size_t)a.E * 4, st, a);
    return hipGetLastError();
  });
  if (e != hipSuccess || !a.groups) return e;
  hipLaunchKernelGGL(sort_kernel, dim3((unsigned)a.groups), dim3(512), sort_lds(a.E), st, a);
  return hipGetLastError();
}

hipError_t launch_moe_sort(const MoeArgs& a, hipStream_t st) {
  if (!a.groups) {
    hipLaunchKernelGGL(sort_one_kernel, dim3(1), dim3(1024), sort_lds(a.E), st, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(count_kernel, dim3((unsigned)a.groups), dim3(256), (size_t)a.E * 4, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(sort_kernel, dim3((unsigned)a.groups), dim3(512), sort_lds(a.E), st, a);
  return hipGetLastError();
}

hipError_t launch_moe_route_backward(const RouteBwdArgs& a, hipStream_t st) {
  return with_lanes(a.f32, a.E, a.k, [&](auto lanes) {
    using W = decltype(lanes);
    const int64_t tokens = 256 / W::LANES, grid = (a.T + tokens - 1) / tokens;
    hipLaunchKernelGGL((route_backward_kernel<W::LANES, W::VPL, W::F32>), dim3((unsigned)grid), dim3(256), 0, st, a);
    return hipGetLastError();
  });
}

// ---------------------------------------------------------- there and back

namespace {

// 2^lx lanes hold 8 2^lx columns of a token; 256 / 2^lx tokens a workgroup.
// UNIFORM (lx >= 6): a wave holds one token, whose rows and weights are scalar loads.
struct Place {
  int64_t t, c;                                // token, first column
  bool there;
};
template <bool UNIFORM>
__device__ __forceinline__ Place place_of(const MoeRowsArgs& a, int lx) {
  Place p;
  const int own = threadIdx.x >> lx;
  p.t = (int64_t)blockIdx.x * (256 >> lx) + (UNIFORM ? __builtin_amdgcn_readfirstlane(own) : own);
  p.c = (((int64_t)blockIdx.y << lx) + (threadIdx.x & ((1 << lx) - 1))) * 8;
  p.there = p.t < a.T && p.c < a.cols;
  return p;
}

// The rows of B slots from j0 on, -1 for none.  All of them are loaded before
// one is used: a load behind the first row's would wait for that row.
template <int B>
__device__ __forceinline__ void rows_of(const MoeRowsArgs& a, const int32_t* row_of, int j0, int* r) {
  const int rows = (int)a.M;
#pragma unroll
  for (int j = 0; j < B; ++j) r[j] = row_of[min(j0 + j, a.k - 1)];
#pragma unroll
  for (int j = 0; j < B; ++j) r[j] = r[j] < rows && j0 + j < a.k ? r[j] : -1;      // negative ones pass through
}

template <int B, bool UNIFORM>
__global__ __launch_bounds__(256) void dispatch_kernel(MoeRowsArgs a, int lx) {
  const Place p = place_of<UNIFORM>(a, lx);
  if (!p.there) return;
  const uint4 v = load16(a.x + p.t * a.ld_x + p.c);
  for (int j0 = 0; j0 < a.k; j0 += B) {
    int r[B];
    rows_of<B>(a, a.row_of + p.t * a.k, j0, r);
#pragma unroll
    for (int j = 0; j < B; ++j)
      if (r[j] >= 0) store16_once(a.to_rows + r[j] * a.ld_to + p.c, v);
  }
}

template <int B, bool UNIFORM, bool WEIGHTS>
__global__ __launch_bounds__(256) void combine_kernel(MoeRowsArgs a, int lx) {
  const Place p = place_of<UNIFORM>(a, lx);
  if (!p.there) return;
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
  for (int j0 = 0; j0 < a.k && a.M > 0; j0 += B) {
    int r[B];
    float w[B];
    uint4 v[B];
    rows_of<B>(a, a.row_of + p.t * a.k, j0, r);
#pragma unroll
    for (int j = 0; j < B; ++j) w[j] = WEIGHTS ? a.weights[p.t * a.k + min(j0 + j, a.k - 1)] : 1.0f;
    // a slot without a row reads row 0, so that all B rows are in flight, and counts
    // as zeros times zero, whatever that row and its weight hold
#pragma unroll
    for (int j = 0; j < B; ++j) v[j] = load16_once(a.rows + max(r[j], 0) * a.ld_rows + p.c);
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const uint32_t keep = r[j] >= 0 ? 0xFFFFFFFFu : 0u;
      const float f = __uint_as_float(__float_as_uint(w[j]) & keep);
      const uint32_t u[4] = {v[j].x & keep, v[j].y & keep, v[j].z & keep, v[j].w & keep};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sum[2 * i] = __builtin_fmaf(f, bf16_lo(u[i]), sum[2 * i]);
        sum[2 * i + 1] = __builtin_fmaf(f, bf16_hi(u[i]), sum[2 * i + 1]);
      }
    }
  }
  store16(a.out + p.t * a.ld_out + p.c, make_uint4(f32x2_to_bf16x2(sum[0], sum[1]), f32x2_to_bf16x2(sum[2], sum[3]),
                                                   f32x2_to_bf16x2(sum[4], sum[5]), f32x2_to_bf16x2(sum[6], sum[7])));
}

// A wave per slot: drow = w dout, dw = dout . row.
__global__ __launch_bounds__(256) void combine_backward_kernel(MoeRowsArgs a) {
  const int lane = threadIdx.x & 63;
  const uint32_t s = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (s >= (uint32_t)(a.T * a.k)) return;      // whole waves leave; slots stay below 2^26
  const int64_t t = s / (uint32_t)a.k, r = a.row_of[s];
  if (r < 0 || r >= a.M) {                     // no row, no gradient
    if (lane == 0) a.dweights[s] = 0.0f;
    return;
  }
  const float w = a.weights[s];
  const uint16_t *g = a.x + t * a.ld_x, *y = a.rows + r * a.ld_rows;
  uint16_t* d = a.to_rows + r * a.ld_to;
  constexpr int B = 4;                         // chunks of a lane in flight
  const int cols = (int)a.cols;
  float dot = 0.0f;
  for (int c0 = 8 * lane; c0 < cols; c0 += 512 * B) {
    uint4 gv[B], yv[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {              // beyond the row: its last chunk, not used
      const int c = min(c0 + 512 * i, cols - 8);
      gv[i] = load16(g + c);
      yv[i] = load16_once(y + c);
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (c0 + 512 * i >= cols) break;
      const uint32_t gu[4] = {gv[i].x, gv[i].y, gv[i].z, gv[i].w}, yu[4] = {yv[i].x, yv[i].y, yv[i].z, yv[i].w};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        dot = __builtin_fmaf(bf16_lo(gu[j]), bf16_lo(yu[j]), dot);
        dot = __builtin_fmaf(bf16_hi(gu[j]), bf16_hi(yu[j]), dot);
        o[j] = f32x2_to_bf16x2(w * bf16_lo(gu[j]), w * bf16_hi(gu[j]));
      }
      store16_once(d + c0 + 512 * i, make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
  dot = lanes_sum<64>(dot);
  if (lane == 0) a.dweights[s] = dot;
}

template <int B_, bool UNIFORM_>
struct Slots {
  static constexpr int B = B_;
  static constexpr bool UNIFORM = UNIFORM_;
};

// Calls f with a Slots: as many slots at once as a token has, up to eight.
template <bool UNIFORM, class F>
void with_slots(int k, F&& f) {
  if (k <= 1) f(Slots<1, UNIFORM>());
  else if (k <= 2) f(Slots<2, UNIFORM>());
  else if (k <= 4) f(Slots<4, UNIFORM>());
  else f(Slots<8, UNIFORM>());
}
template <class F>
void with_slots(int k, int lx, F&& f) {
  if (lx >= 6) with_slots<true>(k, f);
  else with_slots<false>(k, f);
}

int lanes_log2(int64_t cols) {
  int lx = 0;
  while (lx < 8 && (int64_t)8 << lx < cols) ++lx;
  return lx;
}
dim3 rows_grid(const MoeRowsArgs& a, int lx) {
  const int64_t tokens = 256 >> lx, cols = (int64_t)8 << lx;
  return dim3((unsigned)((a.T + tokens - 1) / tokens), (unsigned)((a.cols + cols - 1) / cols));
}

}  // namespace

hipError_t launch_moe_dispatch(const MoeRowsArgs& a, hipStream_t st) {
  const int lx = lanes_log2(a.cols);
  const dim3 grid = rows_grid(a, lx);
  with_slots(a.k, lx, [&](auto w) {
    using W = decltype(w);
    hipLaunchKernelGGL((dispatch_kernel<W::B, W::UNIFORM>), grid, dim3(256), 0, st, a, lx);
  });
  return hipGetLastError();
}

hipError_t launch_moe_combine(const MoeRowsArgs& a, hipStream_t st) {
  const int lx = lanes_log2(a.cols);
  const dim3 grid = rows_grid(a, lx);
  with_slots(a.k, lx, [&](auto w) {
    using W = decltype(w);
    if (a.weights) hipLaunchKernelGGL((combine_kernel<W::B, W::UNIFORM, true>), grid, dim3(256), 0, st, a, lx);
    else hipLaunchKernelGGL((combine_kernel<W::B, W::UNIFORM, false>), grid, dim3(256), 0, st, a, lx);
  });
  return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const MoeRowsArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(combine_backward_kernel, dim3((unsigned)((a.T * a.k + 3) / 4)), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace mxq
