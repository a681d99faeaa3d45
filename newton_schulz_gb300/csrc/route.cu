// Routing of tokens to experts: scores, group cut, top-k, weights; the stable
// counting sort of the chosen (token, slot) pairs by expert; the gradient.
//
// One warp takes one token; lane l holds experts l * EPL .. l * EPL + EPL - 1 in
// registers (EPL experts a lane, a power of two), so a row is read 16 bytes a
// lane, a group of experts is a run of lanes, and the lowest expert among equal
// keys is in the lowest lane that a vote names.  A maximum over the warp is one
// redux instruction on the keys as floats (-inf: not to be chosen).  Bound by
// instruction issue: a token's 4 * experts bytes are little against its scores
// and its top_k rounds.  16384 tokens over 256 experts in 8 groups, top 8: 19 us
// (28.6 with expert e in lane e % 32, a reduction per group); the row plan of
// its 131072 slots 9 us, its counts 2.5 (every block of the plan reads every tile's
// counts: 57 us for 131072 tokens, 1865 for 2^20); the gradient of 16381 tokens
// over 128 experts 6 us.
#include <type_traits>

#include "block.h"
#include "block_ptx.cuh"

namespace muon {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kRouteWarps = 8;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// v[i] = element i of this lane's EPL elements at `at`, `fill` from the n-th on.
// vec: 16-byte aligned where a lane's share is 16 bytes or more (by its size below).
template <int EPL, typename T>
__device__ __forceinline__ void load_share(float (&v)[EPL], const T* at, int n, float fill, bool vec) {
  constexpr int kBytes = EPL * sizeof(T);
  auto value = [](uint32_t w, int half) {
    return sizeof(T) == 4 ? __uint_as_float(w) : __uint_as_float(half ? w & 0xffff0000u : w << 16);
  };
  constexpr int kPer = 4 / sizeof(T);      // elements a word
  if (kBytes >= 4 && vec && n >= EPL) {
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int c = 0; c < kBytes / 16; ++c) {
        const uint4 q = reinterpret_cast<const uint4*>(at)[c];
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4 * kPer; ++i) v[c * 4 * kPer + i] = value(w[i / kPer], i % kPer);
      }
    } else if constexpr (kBytes == 8) {
      const uint2 q = *reinterpret_cast<const uint2*>(at);
      const uint32_t w[2] = {q.x, q.y};
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[i] = value(w[i / kPer], i % kPer);
    } else if constexpr (kBytes == 4) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(at);
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[i] = value(w, i % kPer);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    v[i] = fill;
    if (i < n) {
      if constexpr (sizeof(T) == 4) v[i] = at[i];
      else v[i] = __bfloat162float(at[i]);
    }
  }
}

// As load_share, to memory.
template <int EPL, typename T>
__device__ __forceinline__ void store_share(T* at, const float (&v)[EPL], int n, bool vec) {
  constexpr int kWords = EPL * sizeof(T) / 4;
  if (kWords > 0 && vec && n >= EPL) {
    uint32_t w[kWords > 0 ? kWords : 1];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 4) {
        w[i] = __float_as_uint(v[i]);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    if constexpr (kWords >= 4) {
#pragma unroll
      for (int c = 0; c < kWords / 4; ++c)
        reinterpret_cast<uint4*>(at)[c] = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    } else if constexpr (kWords == 2) {
      *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
    } else {
      *reinterpret_cast<uint32_t*>(at) = w[0];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (i < n) {
      if constexpr (sizeof(T) == 4) at[i] = v[i];
      else at[i] = __float2bfloat16_rn(v[i]);
    }
}

// x[i] = logit of expert lane * EPL + i as read, -inf where there is none.
template <int EPL>
__device__ __forceinline__ void load_logits(float (&x)[EPL], const void* base, int dtype, int64_t row,
                                            int experts, bool vec, int lane) {
  const int first = lane * EPL;
  if (dtype == kDtF32)
    load_share<EPL>(x, static_cast<const float*>(base) + row + first, experts - first, -INFINITY, vec);
  else
    load_share<EPL>(x, static_cast<const __nv_bfloat16*>(base) + row + first, experts - first, -INFINITY, vec);
}
// NaN and +inf become -inf; returns whether one was met.
template <int EPL>
__device__ __forceinline__ bool only_finite(float (&x)[EPL]) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (!(x[i] < INFINITY)) {
      x[i] = -INFINITY;
      bad = true;
    }
  return bad;
}

// Softmax parts: e[i] = exp(x[i] - max), returns their sum (0: every logit is -inf).
template <int EPL>
__device__ __forceinline__ float softmax_parts(const float (&x)[EPL], float (&e)[EPL], float* top) {
  float mx = x[0];
#pragma unroll
  for (int i = 1; i < EPL; ++i) mx = fmaxf(mx, x[i]);
  mx = warp_max(mx);
  *top = mx;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    e[i] = x[i] > -INFINITY ? expf(x[i] - mx) : 0.f;
    sum += e[i];
  }
  return warp_sum(sum);
}

// s = 1 / (1 + exp(-x)) and rest = 1 - s.  From exp(-|x|), so the approximate
// quotient's divisor is in [1, 2] (it gives 0 past 2^126, the scores of logits
// below -87.3), and neither s of a low logit nor rest of a high one is the
// difference of numbers near 1 (from logit 17 on that would be 0): each within
// 3 units of the last place.
__device__ __forceinline__ float sigmoid(float x, float* rest) {
  const float t = expf(-fabsf(x)), r = __fdividef(1.f, 1.f + t), q = t * r;
  *rest = x < 0.f ? r : q;
  return x < 0.f ? q : r;
}
__device__ __forceinline__ float sigmoid(float x) {
  float rest;
  return sigmoid(x, &rest);
}

}  // namespace

template <int EPL>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const __grid_constant__ RouteParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t tok = blockIdx.x * static_cast<int64_t>(kRouteWarps) + (threadIdx.x >> 5);
  ptx::launch_dependents();
  if (tok >= p.tokens) return;
  const int k = p.top_k;
  int32_t my_idx = -1;
  float my_score = 0.f;
  if (!p.mask || p.mask[tok]) {
    const int first = lane * EPL;
    float x[EPL], sc[EPL], key[EPL];
    load_logits<EPL>(x, p.logits, p.dtype, tok * p.stride, p.experts, p.vec, lane);
    if (p.bias) load_share<EPL>(key, p.bias + first, p.experts - first, 0.f, p.bias_vec);
    if (only_finite<EPL>(x)) atomicOr(p.status, kDevNonfinite);
    // every expert's score, where the choice goes by scores
    const bool cut = p.top_groups < p.groups, sum2 = p.group_score == 1;
    const bool by_score = p.bias != nullptr || (cut && sum2);
    float top = 0.f, sum = 0.f;
    if (p.score == 0) {
      sum = softmax_parts<EPL>(x, sc, &top);
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) sc[i] *= inv;
    } else if (by_score) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) sc[i] = sigmoid(x[i]);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float v = p.bias ? sc[i] + key[i] : x[i];
      key[i] = x[i] > -INFINITY && v > -INFINITY ? v : -INFINITY;      // a NaN of the bias: not chosen
    }
    if (cut) {
      const int per = p.experts / p.groups;
      const bool own = sum2 && !p.bias;      // groups ranked by scores, the choice by logits
      auto rank = [&](int i) { return own && key[i] > -INFINITY ? sc[i] : key[i]; };
      // a, b: the two largest of a group
      auto score_of = [&](float a, float b) { return sum2 && b > -INFINITY ? a + b : a; };
      const int run = per / EPL;             // lanes a group
      if (per % EPL == 0 && (run & (run - 1)) == 0) {
        float a = -INFINITY, b = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const float v = rank(i);
          b = fmaxf(b, fminf(a, v));
          a = fmaxf(a, v);
        }
        for (int o = 1; o < run; o <<= 1) {
          const float oa = __shfl_xor_sync(kFull, a, o), ob = __shfl_xor_sync(kFull, b, o);
          b = fmaxf(fmaxf(b, ob), fminf(a, oa));
          a = fmaxf(a, oa);
        }
        float left = score_of(a, b);         // the same in every lane of the group
        bool kept = false;
        for (int j = 0; j < p.top_groups; ++j) {
          const float m = ptx::redux_max(left);
          if (!(m > -INFINITY)) break;
          const int at = __ffs(__ballot_sync(kFull, left == m)) - 1;
          if (((lane ^ at) & ~(run - 1)) == 0) {
            kept = true;
            left = -INFINITY;
          }
        }
        if (!kept) {
#pragma unroll
          for (int i = 0; i < EPL; ++i) key[i] = -INFINITY;
        }
      } else {
        float best[2] = {-INFINITY, -INFINITY};      // this lane: groups lane and 32 + lane
        for (int g = 0; g < p.groups; ++g) {
          float a = -INFINITY, b = -INFINITY;
#pragma unroll
          for (int i = 0; i < EPL; ++i) {
            const int e = first + i - g * per;
            const float v = e >= 0 && e < per ? rank(i) : -INFINITY;
            b = fmaxf(b, fminf(a, v));
            a = fmaxf(a, v);
          }
          const float m1 = ptx::redux_max(a);
          const int owner = __ffs(__ballot_sync(kFull, a == m1)) - 1;
          const float score = score_of(m1, sum2 ? ptx::redux_max(lane == owner ? b : a) : -INFINITY);
          if (lane == (g & 31)) {
            if (g < 32) best[0] = score;
            else best[1] = score;
          }
        }
        uint64_t keep = 0;
        for (int j = 0; j < p.top_groups; ++j) {
          const float m = ptx::redux_max(fmaxf(best[0], best[1]));
          if (!(m > -INFINITY)) break;
          const unsigned lo = __ballot_sync(kFull, best[0] == m), hi = __ballot_sync(kFull, best[1] == m);
          const int g = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);
          keep |= 1ull << g;
          if (lane == (g & 31)) {
            if (g < 32) best[0] = -INFINITY;
            else best[1] = -INFINITY;
          }
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (first + i < p.experts && !((keep >> ((first + i) / per)) & 1)) key[i] = -INFINITY;
      }
    }
    // this lane's two largest keys, lower experts first among equal ones: a lane
    // is looked through again only when it gives its third expert
    float a = -INFINITY, a2 = -INFINITY;
    uint32_t used = 0u;
    int at = 0, at2 = 0;
    auto rescan = [&] {
      a = a2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const float v = (used >> i) & 1u ? -INFINITY : key[i];
        if (v > a) {
          a2 = a;
          at2 = at;
          a = v;
          at = i;
        } else if (v > a2) {
          a2 = v;
          at2 = i;
        }
      }
    };
    rescan();
    bool second = true;      // a2 is the next after a
    for (int j = 0; j < k; ++j) {
      const float m = ptx::redux_max(a);
      if (!(m > -INFINITY)) break;
      const int owner = __ffs(__ballot_sync(kFull, a == m)) - 1;
      const int e = owner * EPL + __shfl_sync(kFull, at, owner);
      if (lane == j) my_idx = e;
      if (lane == owner) {
        used |= 1u << at;
        if (second) {
          a = a2;
          at = at2;
          second = false;
        } else {
          rescan();
          second = true;
        }
      }
    }
    // the chosen experts' scores, each in its lane, from the logit again (in L1)
    if (my_idx >= 0) {
      const int64_t at = tok * p.stride + my_idx;
      const float v = p.dtype == kDtF32 ? static_cast<const float*>(p.logits)[at]
                                        : __bfloat162float(static_cast<const __nv_bfloat16*>(p.logits)[at]);
      my_score = p.score == 0 ? expf(v - top) / sum : sigmoid(v);
    }
  }
  if (p.renorm) {
    const float total = warp_sum(my_score);   // lanes from top_k on hold 0
    my_score = total > 0.f ? my_score / total : 0.f;
  }
  if (lane < k && dbg_ok(my_idx >= -1 && my_idx < p.experts, p.status)) {
    p.idx[tok * k + lane] = my_idx;
    p.weights[tok * k + lane] = my_score * p.scale;
  }
}

template <int EPL>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_grad_kernel(const __grid_constant__ RouteGradParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t tok = blockIdx.x * static_cast<int64_t>(kRouteWarps) + (threadIdx.x >> 5);
  if (tok >= p.tokens) return;
  float x[EPL], sc[EPL], d[EPL];
  load_logits<EPL>(x, p.logits, p.dtype, tok * p.stride, p.experts, p.vec, lane);
  only_finite<EPL>(x);
  float rest[EPL];       // sigmoid: 1 - score
  if (p.score == 0) {
    float top;
    const float sum = softmax_parts<EPL>(x, sc, &top);
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) sc[i] *= inv;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) sc[i] = sigmoid(x[i], &rest[i]);
  }
  int32_t e = -1;
  float dw = 0.f;
  if (lane < p.top_k) {
    e = p.idx[tok * p.top_k + lane];
    dw = p.dweights[tok * p.top_k + lane] * p.scale;
  }
  // each chosen expert's dweight to its lane and register, through shared memory
  constexpr int kPitch = EPL + (EPL >= 4 ? 4 : 1);      // lanes' words in different banks
  __shared__ __align__(16) float s_d[kRouteWarps][32 * kPitch];
  __shared__ uint32_t s_chosen[kRouteWarps][32];
  const int warp = threadIdx.x >> 5;
  float* mine = &s_d[warp][lane * kPitch];
#pragma unroll
  for (int i = 0; i < EPL; ++i) mine[i] = 0.f;
  s_chosen[warp][lane] = 0u;
  __syncwarp();
  if (e >= 0 && e < p.experts && dbg_ok(e / EPL < 32, p.status)) {
    s_d[warp][e / EPL * kPitch + e % EPL] = dw;
    atomicOr(&s_chosen[warp][e / EPL], 1u << (e % EPL));
  }
  __syncwarp();
  const uint32_t chosen = s_chosen[warp][lane];    // bit i: expert lane * EPL + i is chosen
#pragma unroll
  for (int i = 0; i < EPL; ++i) d[i] = mine[i];
  if (p.renorm) {
    // q_i, the chosen scores over their sum; then q_i (d_i - sum d q), where the
    // sum over the chosen is zero, so the full softmax's slope is that as well.
    // The scores are divided, not d: their sum may be as small as 2^-149.
    float total = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      sc[i] = (chosen >> i) & 1u ? sc[i] : 0.f;
      total += sc[i];
    }
    total = warp_sum(total);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      sc[i] = total > 0.f ? sc[i] / total : 0.f;
      dot = fmaf(d[i], sc[i], dot);
    }
    dot = warp_sum(dot);
#pragma unroll
    for (int i = 0; i < EPL; ++i) d[i] = sc[i] * (d[i] - dot) * (p.score == 0 ? 1.f : rest[i]);
  } else if (p.score == 0) {
    float sub = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) sub = fmaf(d[i], sc[i], sub);
    sub = warp_sum(sub);
#pragma unroll
    for (int i = 0; i < EPL; ++i) d[i] = sc[i] * (d[i] - sub);
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) d[i] *= sc[i] * rest[i];
  }
  const int first = lane * EPL;
  const int64_t at = tok * p.dstride + first;
  if (p.dtype == kDtF32) store_share<EPL>(static_cast<float*>(p.dlogits) + at, d, p.experts - first, p.dvec);
  else store_share<EPL>(static_cast<__nv_bfloat16*>(p.dlogits) + at, d, p.experts - first, p.dvec);
}

// ---- plan ------------------------------------------------------------------------------------
namespace {

constexpr int kPlanThreads = 256, kPlanWarps = kPlanThreads / 32;

__device__ __forceinline__ int expert_of(const PlanParams& p, int64_t entry, int64_t end) {
  if (entry >= end) return -1;
  const int e = p.idx[entry];
  return e >= 0 && e < p.experts ? e : -1;
}

}  // namespace

// hist[tile][e]: entries of expert e among the tile's tokens.
__global__ void __launch_bounds__(kPlanThreads) plan_hist_kernel(const __grid_constant__ PlanParams p) {
  extern __shared__ int s_cnt[];
  ptx::launch_dependents();
  for (int e = threadIdx.x; e < p.experts; e += kPlanThreads) s_cnt[e] = 0;
  ptx::wait_dependency();
  __syncthreads();
  const int64_t total = p.tokens * p.top_k;
  const int64_t first = blockIdx.x * static_cast<int64_t>(kPlanTokens) * p.top_k;
  const int64_t end = min(first + static_cast<int64_t>(kPlanTokens) * p.top_k, total);
  for (int64_t i = first + threadIdx.x; i < end; i += kPlanThreads) {
    const int e = expert_of(p, i, end);
    if (e >= 0) atomicAdd(&s_cnt[e], 1);     // a count: no order in it
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += kPlanThreads)
    p.hist[static_cast<int64_t>(blockIdx.x) * p.experts + e] = s_cnt[e];
}

// Rows of one tile: offsets from the column sums of hist, then a stable rank
// within the tile.  Each warp takes a run of consecutive entries; its start
// per expert is the tile's plus the earlier warps' counts.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanParams p) {
  extern __shared__ int smem[];
  int* start = smem;                              // [kPlanWarps][experts]
  int* base = smem + kPlanWarps * p.experts;      // [experts]
  __shared__ int s_scan[kPlanWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.experts;
  const int64_t total = p.tokens * p.top_k;
  const int64_t first = blockIdx.x * static_cast<int64_t>(kPlanTokens) * p.top_k;
  const int64_t end = min(first + static_cast<int64_t>(kPlanTokens) * p.top_k, total);
  for (int i = threadIdx.x; i < kPlanWarps * E; i += kPlanThreads) start[i] = 0;
  ptx::wait_dependency();
  __syncthreads();
  // this tile's counts per warp
  const int64_t run = (end - first + kPlanWarps * 32 - 1) / (kPlanWarps * 32) * 32;
  const int64_t w0 = first + warp * run, w1 = min(w0 + run, end);
  for (int64_t i0 = w0 + lane; i0 < w1; i0 += 128) {      // four loads in flight
    int e[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = expert_of(p, i0 + 32 * j, w1);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (e[j] >= 0) atomicAdd(&start[warp * E + e[j]], 1);
  }
  __syncthreads();
  // expert totals and the entries of earlier tiles; exclusive scan over experts
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += kPlanThreads) {
    const int e = e0 + threadIdx.x;
    int before = 0, all = 0;
    if (e < E) {
      if (p.tiles == 1) {
        for (int w = 0; w < kPlanWarps; ++w) all += start[w * E + e];
      } else {
        for (int b0 = 0; b0 < p.tiles; b0 += 32) {      // 32 loads in flight
          int c[32];
#pragma unroll
          for (int b = 0; b < 32; ++b)
            c[b] = b0 + b < p.tiles ? p.hist[static_cast<int64_t>(b0 + b) * E + e] : 0;
#pragma unroll
          for (int b = 0; b < 32; ++b) {
            all += c[b];
            if (b0 + b < static_cast<int>(blockIdx.x)) before += c[b];
          }
        }
      }
    }
    int v = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kFull, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) s_scan[warp] = v;
    __syncthreads();
    int pre = carry, sum = 0;
    for (int w = 0; w < kPlanWarps; ++w) {
      if (w < warp) pre += s_scan[w];
      sum += s_scan[w];
    }
    const int off = pre + v - all;
    if (e < E) {
      base[e] = off + before;
      if (blockIdx.x == 0) p.offsets[e] = off;
    }
    carry += sum;
    __syncthreads();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) p.offsets[E] = carry;
  // counts -> first rows, in warp order
  for (int e = threadIdx.x; e < E; e += kPlanThreads) {
    int at = base[e];
    for (int w = 0; w < kPlanWarps; ++w) {
      const int c = start[w * E + e];
      start[w * E + e] = at;
      at += c;
    }
  }
  __syncthreads();
  int next = expert_of(p, w0 + lane, w1);
  for (int64_t i0 = w0; i0 < w1; i0 += 32) {
    const int64_t i = i0 + lane;
    const int e = next;
    next = expert_of(p, i + 32, w1);
    const unsigned peers = __match_any_sync(kFull, e);
    int row = -1;
    if (e >= 0) row = start[warp * E + e] + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
    if (e >= 0 && lane == __ffs(peers) - 1) start[warp * E + e] += __popc(peers);
    __syncwarp();
    if (i < w1) {
      p.pos[i] = row;
      if (row >= 0 && dbg_ok(row < total, p.status)) p.src[row] = static_cast<int32_t>(i);
    }
  }
  // entries past the last row
  for (int64_t i = carry + blockIdx.x * static_cast<int64_t>(kPlanThreads) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kPlanThreads)
    p.src[i] = -1;
}

namespace {

template <typename P, typename F>
cudaError_t by_experts(int experts, F&& f) {
  if (experts <= 32) f(std::integral_constant<int, 1>{});
  else if (experts <= 64) f(std::integral_constant<int, 2>{});
  else if (experts <= 128) f(std::integral_constant<int, 4>{});
  else if (experts <= 256) f(std::integral_constant<int, 8>{});
  else if (experts <= 512) f(std::integral_constant<int, 16>{});
  else f(std::integral_constant<int, 32>{});
  return cudaGetLastError();
}

unsigned route_grid(int64_t tokens) { return static_cast<unsigned>((tokens + kRouteWarps - 1) / kRouteWarps); }

}  // namespace

cudaError_t launch_route(const RouteParams& p, cudaStream_t s) {
  return by_experts<RouteParams>(p.experts, [&](auto n) {
    route_kernel<decltype(n)::value><<<route_grid(p.tokens), kRouteWarps * 32, 0, s>>>(p);
  });
}

cudaError_t launch_route_grad(const RouteGradParams& p, cudaStream_t s) {
  return by_experts<RouteGradParams>(p.experts, [&](auto n) {
    route_grad_kernel<decltype(n)::value><<<route_grid(p.tokens), kRouteWarps * 32, 0, s>>>(p);
  });
}

cudaError_t launch_plan_hist(const PlanParams& p, bool early, cudaStream_t s) {
  return launch_after(plan_hist_kernel, p.tiles, kPlanThreads, p.experts * sizeof(int), early, s, p);
}

cudaError_t launch_plan(const PlanParams& p, bool early, cudaStream_t s) {
  // at most (8 + 1) * 1024 counters: 36 KB, under the default limit
  return launch_after(plan_kernel, p.tiles, kPlanThreads, (kPlanWarps + 1) * p.experts * sizeof(int), early, s, p);
}

}  // namespace muon
