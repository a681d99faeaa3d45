// The experts' forward products for a few rows (a decode step of a few tokens):
// matrix-vector products on the CUDA cores, HBM-bound on the weights of the
// experts hit.  A warp takes one output: the gate and up rows of a feature, or
// one column of out over all of a token's slots, 16 bytes a lane and load.  Rows
// of one expert read its weights again, which the rule for taking them counts.
// One token through 8 of 256 experts of [768, 2048] (75 MB): the tile kernels
// took 34 us on 48 and 64 of their 76 CTA pairs' tiles, without the copy and
// the sum over slots that they need besides; these two take 23.
// Everything is fp32 up to out: the activation is no tensor operand here, and
// rounded to bf16 as the tile kernels must it would put out's error at 0.0024 in
// norm instead of the result's own rounding, 0.0017 (and save 2 us of its reads,
// every warp's of the second kernel).
#include "block.h"
#include "block_ptx.cuh"

namespace muon {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Expert of a row: how many experts' rows end at or before it.  `ends`: this
// lane's offsets, all loaded before the first is used.
struct Ends {
  static constexpr int kMost = kRouteMaxExperts / 32;
  int v[kMost];
  __device__ __forceinline__ void load(const int32_t* offsets, int experts, int lane) {
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      v[i] = 0x7fffffff;
      if (32 * i < experts && 32 * i + lane < experts) v[i] = offsets[32 * i + lane + 1];
    }
  }
  __device__ __forceinline__ int expert(int row, int experts) const {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kMost; ++i)
      if (32 * i < experts) n += v[i] <= row;
    return static_cast<int>(__reduce_add_sync(kFull, static_cast<unsigned>(n)));
  }
};

__device__ __forceinline__ float2 two(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ void dot8(const uint4& a, const uint4& b, float2& acc) {
  acc = ptx::fma2(two(a.x), two(b.x), acc);
  acc = ptx::fma2(two(a.y), two(b.y), acc);
  acc = ptx::fma2(two(a.z), two(b.z), acc);
  acc = ptx::fma2(two(a.w), two(b.w), acc);
}
// the same with fp32 a
__device__ __forceinline__ void dot8(const float4& a0, const float4& a1, const uint4& b, float2& acc) {
  acc = ptx::fma2(make_float2(a0.x, a0.y), two(b.x), acc);
  acc = ptx::fma2(make_float2(a0.z, a0.w), two(b.y), acc);
  acc = ptx::fma2(make_float2(a1.x, a1.y), two(b.z), acc);
  acc = ptx::fma2(make_float2(a1.z, a1.w), two(b.w), acc);
}
// weights are read once
__device__ __forceinline__ uint4 ld_once(const __nv_bfloat16* p) {
  return __ldcs(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ uint4 ld(const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); }

}  // namespace

__global__ void __launch_bounds__(kWarps * 32) ex_few_up_kernel(const __grid_constant__ ExFewParams p) {
  const int lane = threadIdx.x & 31;
  const int u = blockIdx.x * kWarps + (threadIdx.x >> 5);      // rows * inner and tokens * hidden fit
  ptx::launch_dependents();
  const int row = u / p.inner, ft = u - row * p.inner;
  if (row >= p.rows) return;
  Ends ends;
  ends.load(p.offsets, p.experts, lane);
  const int32_t s = p.src[row];
  const int e = ends.expert(row, p.experts);
  if (e >= p.experts || s < 0 || s >= p.rows) return;      // past the last row
  if (!dbg_ok(ft < p.inner && s / p.top_k < p.tokens && ft < p.ip, p.status)) return;
  const __nv_bfloat16* x = p.x + (s / p.top_k) * p.xs;
  const __nv_bfloat16* g = p.w_in + (static_cast<int64_t>(e) * 2 * p.inner + ft) * p.hidden;
  const __nv_bfloat16* v = g + static_cast<int64_t>(p.inner) * p.hidden;
  float2 ag = make_float2(0.f, 0.f), au = ag;
  if (p.vec_in) {
    int c = lane * 8;
    for (; c + 3 * 256 < p.hidden; c += 1024) {
      uint4 xv[4], gv[4], uv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        gv[j] = ld_once(g + c + 256 * j);
        uv[j] = ld_once(v + c + 256 * j);
        xv[j] = ld(x + c + 256 * j);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        dot8(xv[j], gv[j], ag);
        dot8(xv[j], uv[j], au);
      }
    }
    for (; c < p.hidden; c += 256) {
      const uint4 xv = ld(x + c);
      dot8(xv, ld_once(g + c), ag);
      dot8(xv, ld_once(v + c), au);
    }
  } else {
    for (int c = lane; c < p.hidden; c += 32) {
      const float xv = __bfloat162float(x[c]);
      ag.x = fmaf(xv, __bfloat162float(g[c]), ag.x);
      au.x = fmaf(xv, __bfloat162float(v[c]), au.x);
    }
  }
  const float gate = warp_sum(ag.x + ag.y), up = warp_sum(au.x + au.y);
  if (lane == 0) {
    p.act[row * p.ip + ft] = gate / (1.f + __expf(-gate)) * up;
    if (p.gu) {
      __nv_bfloat16* o = p.gu + static_cast<int64_t>(row) * 2 * p.inner + ft;
      o[0] = __float2bfloat16_rn(gate);
      o[p.inner] = __float2bfloat16_rn(up);
    }
  }
}

__global__ void __launch_bounds__(kWarps * 32) ex_few_down_kernel(const __grid_constant__ ExFewParams p) {
  const int lane = threadIdx.x & 31;
  const int u = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = u / p.hidden, h = u - t * p.hidden;
  if (t >= p.tokens) return;
  Ends ends;
  ends.load(p.offsets, p.experts, lane);
  int my_row = -1, my_e = 0;
  float my_w = 0.f;
  if (lane < p.top_k) {
    my_row = p.pos[t * p.top_k + lane];
    my_w = p.weights[t * p.top_k + lane];
  }
  for (int j = 0; j < p.top_k; ++j) {
    const int r = __shfl_sync(kFull, my_row, j);
    const int e = ends.expert(r, p.experts);
    if (lane == j) my_e = e;
  }
  if (my_row < 0 || my_row >= p.rows || my_e >= p.experts) {
    my_row = -1;
    my_e = 0;
  }
  if (!dbg_ok(h < p.hidden && t < p.tokens, p.status)) return;
  float acc = 0.f;
  constexpr int kSlots = 4;
  for (int j0 = 0; j0 < p.top_k; j0 += kSlots) {
    const __nv_bfloat16* w[kSlots];
    const float* a[kSlots];
    float wt[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      const int at = (j0 + j) & 31;
      const int r = j0 + j < p.top_k ? __shfl_sync(kFull, my_row, at) : -1;
      const int e = __shfl_sync(kFull, my_e, at);
      wt[j] = __shfl_sync(kFull, my_w, at);
      if (r < 0) wt[j] = 0.f;
      w[j] = r < 0 ? nullptr : p.w_out + (static_cast<int64_t>(e) * p.hidden + h) * p.inner;
      a[j] = p.act + max(r, 0) * p.ip;
    }
    float2 d[kSlots] = {};
    if (p.vec_out) {
      for (int c = lane * 8; c < p.inner; c += 512) {
        uint4 wv[kSlots][2];
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
#pragma unroll
          for (int q = 0; q < 2; ++q)
            if (w[j] && c + 256 * q < p.inner) wv[j][q] = ld_once(w[j] + c + 256 * q);
        ptx::wait_dependency();      // act; the first weights are on their way meanwhile
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float4 av[kSlots][2];
#pragma unroll
          for (int j = 0; j < kSlots; ++j)
            if (w[j] && c + 256 * q < p.inner) {
              const float4* from = reinterpret_cast<const float4*>(a[j] + c + 256 * q);
              av[j][0] = from[0];
              av[j][1] = from[1];
            }
#pragma unroll
          for (int j = 0; j < kSlots; ++j)
            if (w[j] && c + 256 * q < p.inner) dot8(av[j][0], av[j][1], wv[j][q], d[j]);
        }
      }
    } else {
      ptx::wait_dependency();
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (w[j])
          for (int c = lane; c < p.inner; c += 32)
            d[j].x = fmaf(a[j][c], __bfloat162float(w[j][c]), d[j].x);
    }
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (w[j]) acc = fmaf(wt[j], d[j].x + d[j].y, acc);
  }
  acc = warp_sum(acc);
  if (lane == 0) p.out[t * p.outs + h] = __float2bfloat16_rn(acc);
}

cudaError_t launch_ex_few(const ExFewParams& p, cudaStream_t s) {
  const int64_t up = (static_cast<int64_t>(p.rows) * p.inner + kWarps - 1) / kWarps;
  const int64_t down = (p.tokens * p.hidden + kWarps - 1) / kWarps;
  ex_few_up_kernel<<<static_cast<unsigned>(up), kWarps * 32, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(ex_few_down_kernel, static_cast<unsigned>(down), kWarps * 32, 0, true, s, p);
}

}  // namespace muon
