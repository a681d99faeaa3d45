// The experts' products over a routing (see muon_experts_forward): simple
// kernels, right for every size.
//
// Rows are (token, slot) pairs in expert order; expert e has rows
// [offsets[e], offsets[e + 1]).  Every product is a 64 x 64 output tile per
// block, fp32 multiply-adds on operands widened from bf16.
#include "block.h"

namespace muon {

namespace {

constexpr int TS = 64, TK = 16, kThreads = 256;

enum Mode { kGu, kDown, kDa, kDx, kDwIn, kDwOut };

__device__ __forceinline__ int row_begin(const ExpertsParams& p, int e) {
  return static_cast<int>(min(static_cast<int64_t>(max(p.offsets[e], 0)), p.rows));
}

// token of a row, -1 where the plan names none
__device__ __forceinline__ int64_t token_of(const ExpertsParams& p, int64_t row) {
  const int32_t s = p.src[row];
  return s >= 0 && s < p.rows ? s / p.top_k : -1;
}

__device__ __forceinline__ float bf(const __nv_bfloat16* p, int64_t i) { return __bfloat162float(p[i]); }

__device__ __forceinline__ float silu_parts(float g, float* slope) {
  const float s = 1.f / (1.f + expf(-g));
  *slope = s * (1.f + g * (1.f - s));
  return g * s;
}

// Left operand of output row `m`, right operand of output column `n`.
template <int MODE>
__device__ __forceinline__ float left(const ExpertsParams& p, int64_t m, int64_t k, int64_t tok) {
  if (MODE == kGu) return tok >= 0 ? bf(p.x, tok * p.xs + k) : 0.f;
  if (MODE == kDown) return bf(p.act, m * p.inner + k);
  if (MODE == kDa) return tok >= 0 ? bf(p.dout, tok * p.dos + k) : 0.f;
  return bf(p.dgu, m * 2 * p.inner + k);
}
template <int MODE>
__device__ __forceinline__ float right(const ExpertsParams& p, int64_t e, int64_t n, int64_t k) {
  const int64_t H = p.hidden, I = p.inner;
  if (MODE == kGu) return bf(p.w_in, (e * 2 * I + n) * H + k);
  if (MODE == kDown) return bf(p.w_out, (e * H + n) * I + k);
  if (MODE == kDa) return bf(p.w_out, (e * H + k) * I + n);
  return bf(p.w_in, (e * 2 * I + k) * H + n);
}

__device__ __forceinline__ void fma_tile(const float (&a)[TK][TS + 4], const float (&b)[TK][TS + 4],
                                         float (&acc)[4][4], int ty, int tx) {
#pragma unroll
  for (int k = 0; k < TK; ++k) {
    float u[4], v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[i] = a[k][ty * 4 + i];
      v[i] = b[k][tx * 4 + i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(u[i], v[j], acc[i][j]);
  }
}

}  // namespace

// Row products.  blockIdx.y numbers row tiles of all experts, each expert's
// rows starting a tile of its own.
template <int MODE>
__global__ void __launch_bounds__(kThreads) experts_rows_kernel(const __grid_constant__ ExpertsParams p) {
  __shared__ float a[TK][TS + 4], b[TK][TS + 4];
  __shared__ int s_e, s_r0, s_r1;
  if (threadIdx.x == 0) {
    s_e = -1;
    int left_tiles = blockIdx.y;
    for (int e = 0; e < p.experts; ++e) {
      const int r0 = row_begin(p, e), r1 = max(r0, row_begin(p, e + 1));
      const int t = (r1 - r0 + TS - 1) / TS;
      if (left_tiles < t) {
        s_e = e;
        s_r0 = r0 + left_tiles * TS;
        s_r1 = min(s_r0 + TS, r1);
        break;
      }
      left_tiles -= t;
    }
  }
  __syncthreads();
  if (s_e < 0) return;
  const int64_t N = MODE == kGu ? 2 * p.inner : MODE == kDa ? p.inner : p.hidden;
  const int64_t K = MODE == kGu || MODE == kDa ? p.hidden : MODE == kDown ? p.inner : 2 * p.inner;
  const int64_t n0 = blockIdx.x * static_cast<int64_t>(TS);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < K; k0 += TK) {
    for (int i = threadIdx.x; i < TS * TK; i += kThreads) {
      const int r = i / TK, k = i % TK;
      const int64_t row = s_r0 + r;
      const bool ok = row < s_r1 && k0 + k < K;
      const int64_t tok = ok ? token_of(p, row) : -1;
      a[k][r] = ok ? left<MODE>(p, row, k0 + k, tok) : 0.f;
      // weights: neighbouring threads read neighbouring addresses
      constexpr bool kn = MODE == kDa || MODE == kDx;
      const int n = kn ? i % TS : i / TK, kk = kn ? i / TS : i % TK;
      b[kk][n] = n0 + n < N && k0 + kk < K ? right<MODE>(p, s_e, n0 + n, k0 + kk) : 0.f;
    }
    __syncthreads();
    fma_tile(a, b, acc, ty, tx);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t row = s_r0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (row >= s_r1 || n >= N) continue;
      if (MODE == kDa) p.da[row * N + n] = acc[i][j];
      else {
        __nv_bfloat16* o = MODE == kGu ? p.gu : MODE == kDown ? p.y : p.dxr;
        o[row * N + n] = __float2bfloat16_rn(acc[i][j]);
      }
    }
}

// Weight gradients: dw_in[e][f][h] = sum dgu[r][f] x[t][h],
// dw_out[e][h][i] = sum dout[t][h] wact[r][i].
template <int MODE>
__global__ void __launch_bounds__(kThreads) experts_dw_kernel(const __grid_constant__ ExpertsParams p) {
  __shared__ float a[TK][TS + 4], b[TK][TS + 4];
  const int e = blockIdx.z;
  const int64_t M = MODE == kDwIn ? 2 * p.inner : p.hidden, N = MODE == kDwIn ? p.hidden : p.inner;
  const int64_t m0 = blockIdx.y * static_cast<int64_t>(TS), n0 = blockIdx.x * static_cast<int64_t>(TS);
  const int r0 = row_begin(p, e), r1 = row_begin(p, e + 1);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int k0 = r0; k0 < r1; k0 += TK) {
    for (int i = threadIdx.x; i < TS * TK; i += kThreads) {
      const int c = i % TS, k = i / TS;
      const int64_t row = k0 + k;
      const int64_t tok = row < r1 ? token_of(p, row) : -1;
      float u = 0.f, v = 0.f;
      if (tok >= 0) {
        if (m0 + c < M)
          u = MODE == kDwIn ? bf(p.dgu, row * 2 * p.inner + m0 + c) : bf(p.dout, tok * p.dos + m0 + c);
        if (n0 + c < N)
          v = MODE == kDwIn ? bf(p.x, tok * p.xs + n0 + c) : bf(p.wact, row * p.inner + n0 + c);
      }
      a[k][c] = u;
      b[k][c] = v;
    }
    __syncthreads();
    fma_tile(a, b, acc, ty, tx);
    __syncthreads();
  }
  void* o = MODE == kDwIn ? p.dw_in : p.dw_out;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m >= M || n >= N) continue;
      const int64_t at = (e * M + m) * N + n;
      if (p.dw_dt == kDtF32) static_cast<float*>(o)[at] = acc[i][j];
      else static_cast<__nv_bfloat16*>(o)[at] = __float2bfloat16_rn(acc[i][j]);
    }
}

// act = silu(g) u
__global__ void __launch_bounds__(kThreads) experts_act_kernel(const __grid_constant__ ExpertsParams p) {
  const int64_t rows = row_begin(p, p.experts);
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x)
    for (int64_t i = threadIdx.x; i < p.inner; i += kThreads) {
      float slope;
      const float g = bf(p.gu, row * 2 * p.inner + i), u = bf(p.gu, row * 2 * p.inner + p.inner + i);
      p.act[row * p.inner + i] = __float2bfloat16_rn(silu_parts(g, &slope) * u);
    }
}

// dgu, w a and dweights of one row per block turn
__global__ void __launch_bounds__(kThreads) experts_dact_kernel(const __grid_constant__ ExpertsParams p) {
  __shared__ float s_part[kThreads / 32];
  const int64_t rows = row_begin(p, p.experts);
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int32_t s = p.src[row];
    const bool ok = s >= 0 && s < p.rows;
    const float w = ok ? p.weights[s] : 0.f;
    float dot = 0.f;
    for (int64_t i = threadIdx.x; i < p.inner; i += kThreads) {
      float slope;
      const float g = bf(p.gu_in, row * 2 * p.inner + i), u = bf(p.gu_in, row * 2 * p.inner + p.inner + i);
      const float sl = silu_parts(g, &slope), da = p.da[row * p.inner + i];
      dot = fmaf(da, sl * u, dot);
      p.dgu[row * 2 * p.inner + i] = __float2bfloat16_rn(w * da * u * slope);
      p.dgu[row * 2 * p.inner + p.inner + i] = __float2bfloat16_rn(w * da * sl);
      p.wact[row * p.inner + i] = __float2bfloat16_rn(w * sl * u);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = dot;
    __syncthreads();
    if (threadIdx.x == 0 && ok && p.dweights) {
      for (int k = 1; k < kThreads / 32; ++k) dot += s_part[k];
      p.dweights[s] = dot;
    }
    __syncthreads();
  }
}

// out[t] = sum over slots, in slot order
template <bool WEIGHTED>
__global__ void __launch_bounds__(kThreads)
    experts_combine_kernel(const __grid_constant__ ExpertsParams p, const __nv_bfloat16* rows,
                           __nv_bfloat16* out, int64_t outs) {
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x)
    for (int64_t h = threadIdx.x; h < p.hidden; h += kThreads) {
      float v = 0.f;
      for (int j = 0; j < p.top_k; ++j) {
        const int32_t r = p.pos[t * p.top_k + j];
        if (r < 0 || r >= p.rows) continue;
        v = fmaf(WEIGHTED ? p.weights[t * p.top_k + j] : 1.f, bf(rows, r * p.hidden + h), v);
      }
      out[t * outs + h] = __float2bfloat16_rn(v);
    }
}

namespace {

template <int MODE>
cudaError_t rows_launch(const ExpertsParams& p, int64_t n, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((n + TS - 1) / TS),
                  static_cast<unsigned>((p.rows + TS - 1) / TS + p.experts));
  experts_rows_kernel<MODE><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

unsigned many(int64_t n) { return static_cast<unsigned>(n < 4096 ? n : 4096); }

}  // namespace

cudaError_t launch_experts_gu(const ExpertsParams& p, cudaStream_t s) { return rows_launch<kGu>(p, 2 * p.inner, s); }
cudaError_t launch_experts_down(const ExpertsParams& p, cudaStream_t s) { return rows_launch<kDown>(p, p.hidden, s); }
cudaError_t launch_experts_da(const ExpertsParams& p, cudaStream_t s) { return rows_launch<kDa>(p, p.inner, s); }
cudaError_t launch_experts_dx(const ExpertsParams& p, cudaStream_t s) { return rows_launch<kDx>(p, p.hidden, s); }

cudaError_t launch_experts_act(const ExpertsParams& p, cudaStream_t s) {
  experts_act_kernel<<<many(p.rows), kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_experts_dact(const ExpertsParams& p, cudaStream_t s) {
  experts_dact_kernel<<<many(p.rows), kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_experts_dw(const ExpertsParams& p, bool w_out, cudaStream_t s) {
  const int64_t M = w_out ? p.hidden : 2 * p.inner, N = w_out ? p.inner : p.hidden;
  const dim3 grid(static_cast<unsigned>((N + TS - 1) / TS), static_cast<unsigned>((M + TS - 1) / TS),
                  static_cast<unsigned>(p.experts));
  if (w_out) experts_dw_kernel<kDwOut><<<grid, kThreads, 0, s>>>(p);
  else experts_dw_kernel<kDwIn><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_experts_combine(const ExpertsParams& p, const __nv_bfloat16* rows, bool weighted,
                                   __nv_bfloat16* out, int64_t outs, cudaStream_t s) {
  if (weighted) experts_combine_kernel<true><<<many(p.tokens), kThreads, 0, s>>>(p, rows, out, outs);
  else experts_combine_kernel<false><<<many(p.tokens), kThreads, 0, s>>>(p, rows, out, outs);
  return cudaGetLastError();
}

}  // namespace muon
