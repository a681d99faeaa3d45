// Routing of tokens to experts: scores, group cut, top-k, weights; the stable
// counting sort of the chosen (token, slot) pairs by expert; the gradient.
//
// One warp takes one token; expert e sits in lane e % 32, register e / 32.
// A key becomes an unsigned word whose order is the float's (0: not to be
// chosen), so a maximum over the warp is one redux instruction, and the
// lowest expert among equal keys another.  Bound by instruction issue and
// latency: a token's 4 * experts bytes are little against its top_k rounds.
#include <type_traits>

#include "block.h"
#include "block_ptx.cuh"

namespace muon {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kRouteWarps = 8;

__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t b = __float_as_uint(f + 0.f);   // -0 becomes +0: equal keys tie
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

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

// x[i] = logit of expert i * 32 + lane, -inf where there is none or it is
// not finite; returns whether a NaN or +inf was met.
template <int EPL>
__device__ __forceinline__ bool load_logits(float (&x)[EPL], const void* base, int dtype,
                                            int64_t off, int experts, int lane) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * 32 + lane;
    x[i] = -INFINITY;
    if (e < experts) {
      x[i] = dtype == kDtF32
                 ? static_cast<const float*>(base)[off + e]
                 : __bfloat162float(static_cast<const __nv_bfloat16*>(base)[off + e]);
      if (!(x[i] < INFINITY)) {
        x[i] = -INFINITY;
        bad = true;
      }
    }
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

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

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
    float x[EPL], sc[EPL];
    if (load_logits<EPL>(x, p.logits, p.dtype, tok * p.stride, p.experts, lane))
      atomicOr(p.status, kDevNonfinite);
    // every expert's score, where the choice goes by scores
    const bool by_score = p.bias != nullptr || (p.top_groups < p.groups && p.group_score == 1);
    float top = 0.f, sum = 0.f;
    if (p.score == 0) {
      sum = softmax_parts<EPL>(x, sc, &top);
#pragma unroll
      for (int i = 0; i < EPL; ++i) sc[i] = sum > 0.f ? sc[i] / sum : 0.f;
    } else if (by_score) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) sc[i] = sigmoid(x[i]);
    }
    uint32_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = i * 32 + lane;
      const bool alive = x[i] > -INFINITY;
      const float v = p.bias ? sc[i] + (alive ? p.bias[e] : 0.f) : x[i];
      key[i] = alive && v > -INFINITY ? ordered(v) : 0u;
    }
    if (p.top_groups < p.groups) {
      const int per = p.experts / p.groups;
      const bool sum2 = p.group_score == 1;
      // what a group is ranked by, as ordered words
      uint32_t rank[EPL];
#pragma unroll
      for (int i = 0; i < EPL; ++i) rank[i] = sum2 && !p.bias && key[i] ? ordered(sc[i]) : key[i];
      uint32_t best[2] = {0u, 0u};     // this lane: groups lane and 32 + lane
      // a: this lane's largest in the group, b: its second largest
      auto score_of = [&](uint32_t a, uint32_t b) {
        const uint32_t m1 = __reduce_max_sync(kFull, a);
        if (!sum2 || !m1) return m1;
        const int owner = __ffs(__ballot_sync(kFull, a == m1)) - 1;
        const uint32_t m2 = __reduce_max_sync(kFull, lane == owner ? b : a);
        return ordered(m2 ? unordered(m1) + unordered(m2) : unordered(m1));
      };
      uint64_t keep = 0;
      if (per == 32) {
        // register i is group i
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (i < p.groups) {
            const uint32_t score = score_of(rank[i], 0u);
            if (lane == i) best[0] = score;
          }
      } else {
        for (int g = 0; g < p.groups; ++g) {
          uint32_t a = 0u, b = 0u;
#pragma unroll
          for (int i = 0; i < EPL; ++i) {
            const int e = i * 32 + lane - g * per;
            const uint32_t v = e >= 0 && e < per ? rank[i] : 0u;
            b = max(b, min(a, v));
            a = max(a, v);
          }
          const uint32_t score = score_of(a, b);
          if (lane == (g & 31)) {
            if (g < 32) best[0] = score;
            else best[1] = score;
          }
        }
      }
      for (int j = 0; j < p.top_groups; ++j) {
        const uint32_t m = __reduce_max_sync(kFull, max(best[0], best[1]));
        if (!m) break;
        const unsigned lo = __ballot_sync(kFull, best[0] == m), hi = __ballot_sync(kFull, best[1] == m);
        const int g = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);
        keep |= 1ull << g;
        if (lane == (g & 31)) {
          if (g < 32) best[0] = 0u;
          else best[1] = 0u;
        }
      }
      if (per == 32) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (!((keep >> i) & 1)) key[i] = 0u;
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const int e = i * 32 + lane;
          if (e < p.experts && !((keep >> (e / per)) & 1)) key[i] = 0u;
        }
      }
    }
    // this lane's two largest keys, lower experts first among equal ones: a lane
    // is looked through again only when it gives its third expert
    uint32_t a = 0u, a2 = 0u, used = 0u;
    int at = 0, at2 = 0;
    auto rescan = [&] {
      a = a2 = 0u;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const uint32_t v = (used >> i) & 1u ? 0u : key[i];
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
      const uint32_t m = __reduce_max_sync(kFull, a);
      if (!m) break;
      const unsigned who = __ballot_sync(kFull, a == m);
      int owner = __ffs(who) - 1;
      int e = __shfl_sync(kFull, at, owner) * 32 + owner;
      if (who & (who - 1)) {      // equal keys in several lanes
        e = static_cast<int>(__reduce_min_sync(kFull, a == m ? static_cast<uint32_t>(at * 32 + lane) : ~0u));
        owner = e & 31;
      }
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
  if (lane < k) {
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
  load_logits<EPL>(x, p.logits, p.dtype, tok * p.stride, p.experts, lane);
  if (p.score == 0) {
    float top;
    const float sum = softmax_parts<EPL>(x, sc, &top);
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) sc[i] *= inv;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) sc[i] = sigmoid(x[i]);
  }
  int32_t e = -1;
  float dw = 0.f;
  if (lane < p.top_k) {
    e = p.idx[tok * p.top_k + lane];
    dw = p.dweights[tok * p.top_k + lane] * p.scale;
  }
  // each chosen expert's dweight to its lane and register, through shared memory
  __shared__ float s_d[kRouteWarps][EPL * 32];
  __shared__ uint32_t s_chosen[kRouteWarps][32];
  const int warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < EPL; ++i) s_d[warp][i * 32 + lane] = 0.f;
  s_chosen[warp][lane] = 0u;
  __syncwarp();
  if (e >= 0 && e < p.experts) {
    s_d[warp][e] = dw;
    atomicOr(&s_chosen[warp][e & 31], 1u << (e >> 5));
  }
  __syncwarp();
  const uint32_t chosen = s_chosen[warp][lane];    // bit i: expert i * 32 + lane is chosen
#pragma unroll
  for (int i = 0; i < EPL; ++i) d[i] = s_d[warp][i * 32 + lane];
  if (p.renorm) {
    float total = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float q = (chosen >> i) & 1u ? sc[i] : 0.f;
      total += q;
      dot = fmaf(d[i], q, dot);
    }
    total = warp_sum(total);
    dot = warp_sum(dot);
    const float mean = total > 0.f ? dot / total : 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      d[i] = ((chosen >> i) & 1u) && total > 0.f ? (d[i] - mean) / total : 0.f;
  }
  float sub = 0.f;
  if (p.score == 0 && !p.renorm) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) sub = fmaf(d[i], sc[i], sub);
    sub = warp_sum(sub);
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int ei = i * 32 + lane;
    if (ei >= p.experts) continue;
    // renormalised softmax: sum over the chosen of d q is zero, so the full
    // softmax's slope is q d as well
    const float g = p.score == 0 ? sc[i] * (d[i] - sub) : d[i] * sc[i] * (1.f - sc[i]);
    const int64_t at = tok * p.dstride + ei;
    if (p.dtype == kDtF32) static_cast<float*>(p.dlogits)[at] = g;
    else static_cast<__nv_bfloat16*>(p.dlogits)[at] = __float2bfloat16_rn(g);
  }
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
  for (int e = threadIdx.x; e < p.experts; e += kPlanThreads) s_cnt[e] = 0;
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
        for (int b0 = 0; b0 < p.tiles; b0 += 16) {      // 16 loads in flight
          int c[16];
#pragma unroll
          for (int b = 0; b < 16; ++b)
            c[b] = b0 + b < p.tiles ? p.hist[static_cast<int64_t>(b0 + b) * E + e] : 0;
#pragma unroll
          for (int b = 0; b < 16; ++b) {
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
  for (int64_t i0 = w0; i0 < w1; i0 += 32) {
    const int64_t i = i0 + lane;
    const int e = expert_of(p, i, w1);
    const unsigned peers = __match_any_sync(kFull, e);
    int row = -1;
    if (e >= 0) row = start[warp * E + e] + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
    if (e >= 0 && lane == __ffs(peers) - 1) start[warp * E + e] += __popc(peers);
    __syncwarp();
    if (i < w1) {
      p.pos[i] = row;
      if (row >= 0) p.src[row] = static_cast<int32_t>(i);
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

cudaError_t launch_plan_hist(const PlanParams& p, cudaStream_t s) {
  plan_hist_kernel<<<p.tiles, kPlanThreads, p.experts * sizeof(int), s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_plan(const PlanParams& p, bool early, cudaStream_t s) {
  // at most (8 + 1) * 1024 counters: 36 KB, under the default limit
  return launch_after(plan_kernel, p.tiles, kPlanThreads, (kPlanWarps + 1) * p.experts * sizeof(int), early, s, p);
}

}  // namespace muon
