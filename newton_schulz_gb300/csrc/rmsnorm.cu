// RMS norm with the residual's addition and an optional 8-bit output, and its
// gradient.
//
//   h = x + r,  y = gain * h * rstd,  rstd = 1 / sqrt(mean(h^2) + eps)
//   dh = rstd (gain dy - u mean(gain dy u)) + dres,  u = h rstd
//   dgain = sum over rows of dy u
//
// HBM-bound: every input is read once and every output written once; a row
// stays in registers between its statistics and its outputs.  A row is taken
// by `tpr` threads of 8-column chunks (chunk i * tpr + t): part of a warp, or
// a whole block.  All arithmetic is fp32; each output is rounded once.
#include <cuda_fp8.h>

#include <algorithm>

#include "block.h"

namespace muon {

namespace {

// 8 consecutive elements as loaded: bf16 in w[0..3], f32 in w[0..7].
struct Chunk {
  uint32_t w[8];
};

__device__ __forceinline__ void load_chunk(Chunk& c, const void* row, int dt, int col, int cols,
                                           bool vec) {
  if (vec && col + 8 <= cols) {
    if (dt == kDtBf16) {
      const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(row) + col);
      c.w[0] = a.x; c.w[1] = a.y; c.w[2] = a.z; c.w[3] = a.w;
    } else {
      const float* p = static_cast<const float*>(row) + col;
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      const uint4 b = *reinterpret_cast<const uint4*>(p + 4);
      c.w[0] = a.x; c.w[1] = a.y; c.w[2] = a.z; c.w[3] = a.w;
      c.w[4] = b.x; c.w[5] = b.y; c.w[6] = b.z; c.w[7] = b.w;
    }
    return;
  }
  if (dt == kDtBf16) {
    const uint16_t* p = static_cast<const uint16_t*>(row) + col;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = col + 2 * j < cols ? p[2 * j] : 0u;
      const uint32_t hi = col + 2 * j + 1 < cols ? p[2 * j + 1] : 0u;
      c.w[j] = lo | (hi << 16);
    }
  } else {
    const uint32_t* p = static_cast<const uint32_t*>(row) + col;
#pragma unroll
    for (int j = 0; j < 8; ++j) c.w[j] = col + j < cols ? p[j] : 0u;
  }
}

__device__ __forceinline__ void to_float(const Chunk& c, int dt, float (&v)[8]) {
  if (dt == kDtBf16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(c.w[j] << 16);
      v[2 * j + 1] = __uint_as_float(c.w[j] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(c.w[j]);
  }
}

__device__ __forceinline__ void store_chunk(void* row, int dt, int col, int cols, bool vec,
                                            const float (&v)[8]) {
  const bool full = vec && col + 8 <= cols;
  if (dt == kDtBf16) {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(row) + col;
    if (full) {
      uint4 u;
      __nv_bfloat162* q = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      *reinterpret_cast<uint4*>(p) = u;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < cols) p[j] = __float2bfloat16_rn(v[j]);
    }
  } else if (dt == kDtF32) {
    float* p = static_cast<float*>(row) + col;
    if (full) {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < cols) p[j] = v[j];
    }
  } else {
    __nv_fp8_storage_t* p = static_cast<__nv_fp8_storage_t*>(row) + col;
    if (full) {
      uint2 u;
      __nv_fp8x2_storage_t* q = reinterpret_cast<__nv_fp8x2_storage_t*>(&u);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        q[j] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * j], v[2 * j + 1]), __NV_SATFINITE, __NV_E4M3);
      *reinterpret_cast<uint2*>(p) = u;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < cols) p[j] = __nv_cvt_float_to_fp8(v[j], __NV_SATFINITE, __NV_E4M3);
    }
  }
}

__device__ __forceinline__ const char* row_ptr(const void* base, int dt, int64_t row, int64_t stride) {
  return static_cast<const char*>(base) + row * stride * (dt == kDtF32 ? 4 : dt == kDtBf16 ? 2 : 1);
}
__device__ __forceinline__ char* row_ptr(void* base, int dt, int64_t row, int64_t stride) {
  return static_cast<char*>(base) + row * stride * (dt == kDtF32 ? 4 : dt == kDtBf16 ? 2 : 1);
}

// Sum or maximum over the tpr threads of a row, the same value in all of
// them.  tpr <= 32: a power of two, lanes of one warp.  Otherwise the whole
// block, through `slots` (32 floats, not reused before another barrier).
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, int tpr, float* slots) {
  for (int o = min(tpr, 32) >> 1; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, w) : v + w;
  }
  if (tpr <= 32) return v;
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  const int n = tpr >> 5;
  float r = slots[0];
  for (int i = 1; i < n; ++i) r = MAX ? fmaxf(r, slots[i]) : r + slots[i];
  return r;
}

}  // namespace

template <int NV>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512)
    rmsnorm_kernel(const __grid_constant__ NormParams p, int tpr) {
  __shared__ float s_sum[32], s_max[32];
  const int t = static_cast<int>(threadIdx.x) % tpr;
  const int64_t row_raw = blockIdx.x * static_cast<int64_t>(blockDim.x / tpr) + threadIdx.x / tpr;
  // spare threads of the last block repeat the last row without storing
  const bool live = row_raw < p.rows;
  const int64_t row = live ? row_raw : p.rows - 1;
  const bool vec = p.vec != 0;
  const char* xr = row_ptr(p.x, p.x_dt, row, p.xs);
  Chunk cx[NV], cr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * tpr + t) * 8;
    if (col < p.cols) load_chunk(cx[i], xr, p.x_dt, col, p.cols, vec);
  }
  if (p.r_dt != kDtNone) {
    const char* rr = row_ptr(p.res, p.r_dt, row, p.rs);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * tpr + t) * 8;
      if (col < p.cols) load_chunk(cr[i], rr, p.r_dt, col, p.cols, vec);
    }
  }
  float v[NV][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if ((i * tpr + t) * 8 < p.cols) {
      to_float(cx[i], p.x_dt, v[i]);
      if (p.r_dt != kDtNone) {
        float r[8];
        to_float(cr[i], p.r_dt, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += r[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
  }
  if (p.h_dt != kDtNone && live) {
    char* hr = row_ptr(p.h, p.h_dt, row, p.hs);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * tpr + t) * 8;
      if (col < p.cols) store_chunk(hr, p.h_dt, col, p.cols, vec, v[i]);
    }
  }
  ss = row_reduce<false>(ss, tpr, s_sum);
  const float rstd = 1.f / sqrtf(ss / static_cast<float>(p.cols) + p.eps);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * tpr + t) * 8;
    float g[8];
    if (p.g_dt != kDtNone && col < p.cols) {
      Chunk cg;
      load_chunk(cg, p.gain, p.g_dt, col, p.cols, vec);
      to_float(cg, p.g_dt, g);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = 1.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] = v[i][j] * rstd * g[j];
      if (p.group_chunks == 0) top = fmaxf(top, fabsf(v[i][j]));
    }
  }
  char* yr = row_ptr(p.y, p.y_dt, row, p.ys);
  if (p.y_dt != kDtE4m3) {
    if (live) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * tpr + t) * 8;
        if (col < p.cols) store_chunk(yr, p.y_dt, col, p.cols, vec, v[i]);
      }
    }
    return;
  }
  if (p.group_chunks == 0) top = fmaxf(row_reduce<true>(top, tpr, s_max), 1e-12f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * tpr + t, col = c * 8;
    if (p.group_chunks != 0) {
      // 16 chunks (128 columns) lie in 16 consecutive lanes: tpr is a multiple of 16
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[i][j]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      top = fmaxf(m, 1e-12f);
    }
    if (live && col < p.cols) {
      const float k = 448.f / top;
      float q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = v[i][j] * k;
      store_chunk(yr, kDtE4m3, col, p.cols, vec, q);
      const int piece = p.group_chunks ? c / p.group_chunks : 0;
      if (c == piece * p.group_chunks) p.scales[row * p.n_scales + piece] = top / 448.f;
    }
  }
}

// Gradient: row slot s takes rows s, s + slots, ...; its share of dgain stays
// in registers until the end.
template <int NV>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512)
    rmsnorm_grad_kernel(const __grid_constant__ NormGradParams p, int tpr) {
  __shared__ float s_a[2][32], s_b[2][32];
  const int t = static_cast<int>(threadIdx.x) % tpr;
  const int per = blockDim.x / tpr;
  const int slot = blockIdx.x * per + threadIdx.x / tpr;
  const int slots = gridDim.x * per;
  const bool vec = p.vec != 0;
  float acc[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  // every thread of a block makes the same number of turns (block barriers)
  const int64_t turns = (p.rows + slots - 1) / slots;
  int par = 0;
  for (int64_t k = 0; k < turns; ++k, par ^= 1) {
    const int64_t row_raw = slot + k * slots;
    const bool live = row_raw < p.rows;
    const int64_t row = live ? row_raw : p.rows - 1;
    const char* dyr = row_ptr(p.dy, p.dy_dt, row, p.dys);
    const char* hr = row_ptr(p.h, p.h_dt, row, p.hs);
    Chunk cd[NV], ch[NV], cs[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * tpr + t) * 8;
      if (col < p.cols) load_chunk(cd[i], dyr, p.dy_dt, col, p.cols, vec);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * tpr + t) * 8;
      if (col < p.cols) load_chunk(ch[i], hr, p.h_dt, col, p.cols, vec);
    }
    if (p.dr_dt != kDtNone) {
      const char* dr = row_ptr(p.dres, p.dr_dt, row, p.drs);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * tpr + t) * 8;
        if (col < p.cols) load_chunk(cs[i], dr, p.dr_dt, col, p.cols, vec);
      }
    }
    float d[NV][8], h[NV][8];
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * tpr + t) * 8;
      if (col < p.cols) {
        to_float(cd[i], p.dy_dt, d[i]);
        to_float(ch[i], p.h_dt, h[i]);
        float g[8];
        if (p.g_dt != kDtNone) {
          Chunk cg;
          load_chunk(cg, p.gain, p.g_dt, col, p.cols, vec);
          to_float(cg, p.g_dt, g);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] = 1.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ss = fmaf(h[i][j], h[i][j], ss);
          dot = fmaf(d[i][j] * g[j], h[i][j], dot);
        }
      }
    }
    ss = row_reduce<false>(ss, tpr, s_a[par]);
    dot = row_reduce<false>(dot, tpr, s_b[par]);
    const float n = static_cast<float>(p.cols);
    const float rstd = 1.f / sqrtf(ss / n + p.eps);
    const float m = dot * rstd / n;      // mean(gain dy u)
    char* out = row_ptr(p.dh, p.dh_dt, row, p.dhs);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * tpr + t) * 8;
      if (col < p.cols && live) {
        float g[8], s[8], o[8];
        if (p.g_dt != kDtNone) {
          Chunk cg;
          load_chunk(cg, p.gain, p.g_dt, col, p.cols, vec);
          to_float(cg, p.g_dt, g);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] = 1.f;
        }
        if (p.dr_dt != kDtNone) to_float(cs[i], p.dr_dt, s);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float u = h[i][j] * rstd;
          acc[i][j] = fmaf(d[i][j], u, acc[i][j]);
          o[j] = rstd * (d[i][j] * g[j] - u * m) + (p.dr_dt != kDtNone ? s[j] : 0.f);
        }
        store_chunk(out, p.dh_dt, col, p.cols, vec, o);
      }
    }
  }
  if (p.part) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * tpr + t) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < p.cols) p.part[static_cast<int64_t>(slot) * p.cols + col + j] = acc[i][j];
    }
  }
}

// dgain[c] = sum over slots of part[slot][c], slots in a fixed order.
__global__ void __launch_bounds__(256) rmsnorm_dgain_kernel(const float* part, int slots, int cols,
                                                            float* dgain) {
  __shared__ float s[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31);
  const int g = threadIdx.x >> 5;
  float v = 0.f;
  if (c < cols)
    for (int k = g; k < slots; k += 8) v += part[static_cast<int64_t>(k) * cols + c];
  s[g][threadIdx.x & 31] = v;
  __syncthreads();
  if (g == 0 && c < cols) {
#pragma unroll
    for (int k = 1; k < 8; ++k) v += s[k][threadIdx.x & 31];
    dgain[c] = v;
  }
}

namespace {

int pow2_at_least(int n) {
  int v = 1;
  while (v < n) v *= 2;
  return v;
}

// Threads per row for NV chunks a thread: a power of two up to a warp, else
// whole warps.
int threads_per_row(int cols, int nv, int least) {
  const int chunks = (cols + 7) / 8;
  const int t = std::max((chunks + nv - 1) / nv, least);
  return t <= 32 ? pow2_at_least(t) : (t + 31) / 32 * 32;
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, int sms, cudaStream_t s) {
  // Few rows: one chunk a thread, the shortest chain.  Many: four loads in
  // flight a thread.
  const int chunks = (p.cols + 7) / 8;
  const int nv = p.rows <= 4 * sms && chunks <= 1024 ? 1 : chunks <= 2048 ? 4 : 8;
  const int tpr = threads_per_row(p.cols, nv, 16);
  const int block = tpr > 32 ? tpr : 128;
  const int64_t grid = (p.rows + block / tpr - 1) / (block / tpr);
  const dim3 g(static_cast<unsigned>(grid));
  if (nv == 1) rmsnorm_kernel<1><<<g, block, 0, s>>>(p, tpr);
  else if (nv == 4) rmsnorm_kernel<4><<<g, block, 0, s>>>(p, tpr);
  else rmsnorm_kernel<8><<<g, block, 0, s>>>(p, tpr);
  return cudaGetLastError();
}

namespace {

struct GradShape {
  int nv, tpr, block, grid;
};

GradShape grad_shape(const NormGradParams& p, int sms) {
  GradShape g;
  const int chunks = (p.cols + 7) / 8;
  g.nv = p.rows <= 4 * sms && chunks <= 1024 ? 1 : chunks <= 1024 ? 2 : chunks <= 2048 ? 4 : 8;
  g.tpr = threads_per_row(p.cols, g.nv, 8);
  g.block = g.tpr > 32 ? g.tpr : 128;
  const int per = g.block / g.tpr;
  const int64_t most = static_cast<int64_t>(sms) * std::max(1, 512 / g.block) * per;
  // rows a slot, then no more slots than that needs
  const int64_t turns = (p.rows + most - 1) / most;
  const int64_t slots = (p.rows + turns - 1) / turns;
  g.grid = static_cast<int>((slots + per - 1) / per);
  return g;
}

}  // namespace

int norm_grad_slots(const NormGradParams& p, int sms) {
  const GradShape g = grad_shape(p, sms);
  return g.grid * (g.block / g.tpr);
}

cudaError_t launch_norm_grad(const NormGradParams& p, int sms, cudaStream_t s) {
  const GradShape g = grad_shape(p, sms);
  if (g.nv == 1) rmsnorm_grad_kernel<1><<<g.grid, g.block, 0, s>>>(p, g.tpr);
  else if (g.nv == 2) rmsnorm_grad_kernel<2><<<g.grid, g.block, 0, s>>>(p, g.tpr);
  else if (g.nv == 4) rmsnorm_grad_kernel<4><<<g.grid, g.block, 0, s>>>(p, g.tpr);
  else rmsnorm_grad_kernel<8><<<g.grid, g.block, 0, s>>>(p, g.tpr);
  return cudaGetLastError();
}

cudaError_t launch_norm_dgain(const float* part, int slots, int cols, float* dgain, cudaStream_t s) {
  rmsnorm_dgain_kernel<<<(cols + 31) / 32, 256, 0, s>>>(part, slots, cols, dgain);
  return cudaGetLastError();
}

}  // namespace muon
