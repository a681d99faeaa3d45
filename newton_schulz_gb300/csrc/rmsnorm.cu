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
// a whole block.  All arithmetic is fp32; each output is rounded once.  The
// reciprocal root and the codes' factor are CUDA's approximate ones (within 2
// units of the last place): with 256 threads a row, exact divisions by each of
// them were a fifth of the instructions.
//
// Of the measured copy rate: 16384 x 8192 bf16 with a residual 172 us, 0.92
// (a ring of bulk copies 184 us); its gradient at 16384 x 4096 80 us, 0.98, and
// 4 us for the gains' sums; 4099 x 2048 into e4m3 per 128 columns 19 us, 0.71: its
// registers leave 25 warps an SM, too few for the loads' and conversions' latency.
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "block.h"
#include "block_ptx.cuh"

namespace muon {

namespace {

constexpr int kNormStages = 8;      // most stages of the gradient's ring
constexpr int kNormRingBytes = 100 * 1024;

// 8 consecutive elements as loaded: bf16 in w[0..3], f32 in w[0..7].  A row
// waits for its statistics in this form: where every input is bf16 (WIDE
// false) that is half the registers, so twice the loads in flight on an SM.
template <bool WIDE>
struct Chunk {
  uint32_t w[WIDE ? 8 : 4];
};

template <bool WIDE>
__device__ __forceinline__ void load_chunk(Chunk<WIDE>& c, const void* row, int dt, int col, int cols,
                                           bool vec) {
  if (!WIDE) dt = kDtBf16;
  if (vec && col + 8 <= cols) {
    if (dt == kDtBf16) {
      const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(row) + col);
      c.w[0] = a.x; c.w[1] = a.y; c.w[2] = a.z; c.w[3] = a.w;
    } else {
      const float* p = static_cast<const float*>(row) + col;
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      const uint4 b = *reinterpret_cast<const uint4*>(p + 4);
      c.w[0] = a.x; c.w[1] = a.y; c.w[2] = a.z; c.w[3] = a.w;
      if constexpr (WIDE) {
        c.w[4] = b.x; c.w[5] = b.y; c.w[6] = b.z; c.w[7] = b.w;
      }
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
    for (int j = 0; j < (WIDE ? 8 : 4); ++j) c.w[j] = col + j < cols ? p[j] : 0u;
  }
}

template <bool WIDE>
__device__ __forceinline__ void to_float(const Chunk<WIDE>& c, int dt, float (&v)[8]) {
  if (!WIDE || dt == kDtBf16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(c.w[j] << 16);
      v[2 * j + 1] = __uint_as_float(c.w[j] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(c.w[WIDE ? j : 0]);
  }
}

template <bool WIDE>
__device__ __forceinline__ void to_float2(const Chunk<WIDE>& c, int dt, float2 (&v)[4]) {
  float x[8];
  to_float<WIDE>(c, dt, x);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = make_float2(x[2 * j], x[2 * j + 1]);
}

// gain[col .. col + 8), ones where there is none
__device__ __forceinline__ void load_gain(float (&g)[8], const void* gain, int dt, int col, int cols,
                                          bool vec) {
  if (dt != kDtNone && col < cols) {
    Chunk<true> c;
    load_chunk<true>(c, gain, dt, col, cols, vec);
    to_float<true>(c, dt, g);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = 1.f;
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

// Two sums at once, one barrier.
__device__ __forceinline__ void row_reduce2(float& a, float& b, int tpr, float* sa, float* sb) {
  for (int o = min(tpr, 32) >> 1; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if (tpr <= 32) return;
  if ((threadIdx.x & 31) == 0) {
    sa[threadIdx.x >> 5] = a;
    sb[threadIdx.x >> 5] = b;
  }
  __syncthreads();
  const int n = tpr >> 5;
  a = sa[0];
  b = sb[0];
  for (int i = 1; i < n; ++i) {
    a += sa[i];
    b += sb[i];
  }
}

// What e4m3 values are multiplied by for their codes.  The approximate quotient
// gives 0 for divisors past 2^126; a scale, the largest magnitude over 448, stays
// below that, the magnitude itself does not.
__device__ __forceinline__ float code_factor(float scale) { return __fdividef(1.f, scale); }

}  // namespace

// One row from its loaded chunks: statistics, h, y.
template <int NV, bool WIDE>
__device__ __forceinline__ void norm_row(const NormParams& p, const Chunk<WIDE> (&cx)[NV],
                                         const Chunk<WIDE> (&cr)[NV], int64_t row, bool live, int t, int tpr,
                                         float* s_sum, float* s_max) {
  const bool vec = p.vec != 0, has_res = p.r_dt != kDtNone;
  // h of chunk i, recomputed where it is needed
  auto sum = [&](int i, float2 (&v)[4]) {
    if ((i * tpr + t) * 8 >= p.cols) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = make_float2(0.f, 0.f);
      return;
    }
    to_float2<WIDE>(cx[i], p.x_dt, v);
    if (has_res) {
      float2 r[4];
      to_float2<WIDE>(cr[i], p.r_dt, r);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = ptx::add2(v[j], r[j]);
    }
  };
  auto flat = [](const float2 (&v)[4], float (&o)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[2 * j] = v[j].x;
      o[2 * j + 1] = v[j].y;
    }
  };
  char* hr = p.h_dt != kDtNone ? row_ptr(p.h, p.h_dt, row, p.hs) : nullptr;
  float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * tpr + t) * 8;
    float2 v[4];
    sum(i, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) s2 = ptx::fma2(v[j], v[j], s2);
    if (hr && live && col < p.cols) {
      float o[8];
      flat(v, o);
      store_chunk(hr, p.h_dt, col, p.cols, vec, o);
    }
  }
  const float ss = row_reduce<false>(s2.x + s2.y, tpr, s_sum);
  const float rstd = rsqrtf(fmaf(ss, p.inv_cols, p.eps));
  const float2 r2 = make_float2(rstd, rstd);
  // gain * h * rstd of chunk i
  auto scaled = [&](int i, float (&o)[8]) {
    float2 v[4];
    float g[8];
    sum(i, v);
    load_gain(g, p.gain, p.g_dt, (i * tpr + t) * 8, p.cols, vec);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = ptx::mul2(ptx::mul2(v[j], r2), make_float2(g[2 * j], g[2 * j + 1]));
    flat(v, o);
  };
  char* yr = row_ptr(p.y, p.y_dt, row, p.ys);
  const bool e4m3 = p.y_dt == kDtE4m3;
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * tpr + t, col = c * 8;
    float v[8];
    scaled(i, v);
    if (!e4m3) {
      if (live && col < p.cols) store_chunk(yr, p.y_dt, col, p.cols, vec, v);
      continue;
    }
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
    if (!p.grouped) {
      top = fmaxf(top, m);
      continue;
    }
    // 16 chunks (128 columns) lie in 16 consecutive lanes: tpr is a multiple of 16
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = fmaxf(m, 1e-12f);
    if (live && col < p.cols) {
      const float scale = m * (1.f / 448.f), k = code_factor(scale);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= k;
      store_chunk(yr, kDtE4m3, col, p.cols, vec, v);
      if ((c & 15) == 0) p.scales[row * p.n_scales + (c >> 4)] = scale;
    }
  }
  if (!e4m3 || p.grouped) return;
  // one scale for the row
  top = fmaxf(row_reduce<true>(top, tpr, s_max), 1e-12f);
  const float scale = top * (1.f / 448.f), k = code_factor(scale);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * tpr + t) * 8;
    if (!live || col >= p.cols) continue;
    float v[8];
    scaled(i, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= k;
    store_chunk(yr, kDtE4m3, col, p.cols, vec, v);
    if (col == 0) p.scales[row] = scale;
  }
}

template <int NV, bool WIDE>
__global__ void __launch_bounds__(NV == 1 ? 1024 : NV == 8 ? 512 : 256, NV == 2 ? 3 : NV == 4 ? (WIDE ? 2 : 3) : 1)
    rmsnorm_kernel(const __grid_constant__ NormParams p, int tpr) {
  __shared__ float s_sum[32], s_max[32];
  const int t = static_cast<int>(threadIdx.x) % tpr;
  const int64_t row_raw = blockIdx.x * static_cast<int64_t>(blockDim.x / tpr) + threadIdx.x / tpr;
  // spare threads of the last block repeat the last row without storing
  const bool live = row_raw < p.rows;
  const int64_t row = live ? row_raw : p.rows - 1;
  const bool vec = p.vec != 0;
  const bool has_res = p.r_dt != kDtNone;
  // a row's chunks cover it, and its threads are one warp's or the block's
  if (!dbg_ok(row >= 0 && static_cast<int64_t>(NV) * tpr * 8 >= p.cols &&
                  (tpr <= 32 ? 32 % tpr == 0 : tpr == static_cast<int>(blockDim.x)), p.status))
    return;
  const char* xr = row_ptr(p.x, p.x_dt, row, p.xs);
  const char* rr = has_res ? row_ptr(p.res, p.r_dt, row, p.rs) : xr;
  Chunk<WIDE> cx[NV], cr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * tpr + t) * 8;
    if (col < p.cols) load_chunk<WIDE>(cx[i], xr, p.x_dt, col, p.cols, vec);
  }
  if (has_res) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * tpr + t) * 8;
      if (col < p.cols) load_chunk<WIDE>(cr[i], rr, p.r_dt, col, p.cols, vec);
    }
  }
  norm_row<NV, WIDE>(p, cx, cr, row, live, t, tpr, s_sum, s_max);
}

__device__ __forceinline__ bool wait_bounded(uint64_t* full, uint32_t parity, unsigned* status,
                                             unsigned long long timeout_ns) {
  const uint32_t bar = ptx::smem_u32(full);
  bool ok = ptx::mbar_try_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = ptx::globaltimer();
    while (!(ok = ptx::mbar_try_wait(bar, parity)))
      if (ptx::globaltimer() - t0 > timeout_ns) {
        atomicOr(status, kDevTimeout);
        break;
      }
  }
  return ok;
}
// Of a whole block on one of its ring's stages; false: gave up.
__device__ __forceinline__ bool ring_wait(uint64_t* full, uint32_t parity, unsigned* status,
                                          unsigned long long timeout_ns) {
  return !__syncthreads_or(!wait_bounded(full, parity, status, timeout_ns));
}
// After a wait that gave up at stage s: the copies still on their way (of `left`
// rows at most) end before the block's memory does.
__device__ __noinline__ void ring_drain(uint64_t* full, int stages, int s, uint32_t phase, int64_t left,
                                        unsigned* status, unsigned long long timeout_ns) {
  for (int k = 0; k < stages && k < left; ++k) {
    const int at = s + k < stages ? s + k : s + k - stages;
    wait_bounded(&full[at], phase ^ (s + k < stages ? 0u : 1u), status, timeout_ns);
  }
}

// Gradient: row slot s takes rows s, s + slots, ...; its share of dgain stays
// in registers until the end.
template <int NV, bool WIDE>
__global__ void __launch_bounds__(NV == 1 ? 1024 : NV == 8 ? 512 : 256, NV == 2 ? (WIDE ? 2 : 3) : 1)
    rmsnorm_grad_kernel(const __grid_constant__ NormGradParams p, int tpr) {
  __shared__ float s_a[2][32], s_b[2][32];
  const int t = static_cast<int>(threadIdx.x) % tpr;
  const int per = blockDim.x / tpr;
  const int slot = blockIdx.x * per + threadIdx.x / tpr;
  const int slots = gridDim.x * per;
  const bool vec = p.vec != 0;
  const bool has_res = p.dr_dt != kDtNone;
  if (!dbg_ok(static_cast<int64_t>(NV) * tpr * 8 >= p.cols &&
                  (tpr <= 32 ? 32 % tpr == 0 : tpr == static_cast<int>(blockDim.x)), p.status))
    return;
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
    const char* sr = has_res ? row_ptr(p.dres, p.dr_dt, row, p.drs) : hr;
    Chunk<WIDE> cd[NV], ch[NV], cs[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * tpr + t) * 8;
      if (col < p.cols) {
        load_chunk<WIDE>(cd[i], dyr, p.dy_dt, col, p.cols, vec);
        load_chunk<WIDE>(ch[i], hr, p.h_dt, col, p.cols, vec);
      }
    }
    if (has_res) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * tpr + t) * 8;
        if (col < p.cols) load_chunk<WIDE>(cs[i], sr, p.dr_dt, col, p.cols, vec);
      }
    }
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * tpr + t) * 8;
      if (col < p.cols) {
        float d[8], h[8], g[8];
        to_float<WIDE>(cd[i], p.dy_dt, d);
        to_float<WIDE>(ch[i], p.h_dt, h);
        load_gain(g, p.gain, p.g_dt, col, p.cols, vec);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ss = fmaf(h[j], h[j], ss);
          dot = fmaf(d[j] * g[j], h[j], dot);
        }
      }
    }
    row_reduce2(ss, dot, tpr, s_a[par], s_b[par]);
    const float rstd = rsqrtf(fmaf(ss, p.inv_cols, p.eps));
    const float m = dot * rstd * p.inv_cols;      // mean(gain dy u)
    char* out = row_ptr(p.dh, p.dh_dt, row, p.dhs);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * tpr + t) * 8;
      if (col < p.cols && live) {
        float d[8], h[8], g[8], s[8], o[8];
        to_float<WIDE>(cd[i], p.dy_dt, d);
        to_float<WIDE>(ch[i], p.h_dt, h);
        load_gain(g, p.gain, p.g_dt, col, p.cols, vec);
        if (has_res) to_float<WIDE>(cs[i], p.dr_dt, s);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float u = h[j] * rstd;
          acc[i][j] = fmaf(d[j], u, acc[i][j]);
          o[j] = rstd * (d[j] * g[j] - u * m) + (has_res ? s[j] : 0.f);
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

// Gradient over many long rows: a block per row slot, its next rows in flight
// as bulk copies into a shared-memory ring, so the loads need no registers and
// never wait for a row's reduction; the gains stay in registers.  A stage is
// free again once the reduction's barrier is passed (every thread has read
// its chunks by then).
template <int NV, bool WIDE>
__global__ void __launch_bounds__(256, 2)
    rmsnorm_grad_ring_kernel(const __grid_constant__ NormGradParams p, int stages) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float s_a[2][32], s_b[2][32];
  __shared__ uint64_t full[kNormStages];
  const int t = threadIdx.x, tpr = blockDim.x;
  const bool has_res = p.dr_dt != kDtNone;
  const uint32_t bd = p.cols * (p.dy_dt == kDtF32 ? 4 : 2), bh = p.cols * (p.h_dt == kDtF32 ? 4 : 2),
                 bs = has_res ? p.cols * (p.dr_dt == kDtF32 ? 4 : 2) : 0, bytes = bd + bh + bs;
  const uint32_t pitch = (bytes + 127) / 128 * 128;
  const int step = gridDim.x, rows = static_cast<int>(p.rows);
  auto fetch = [&](int64_t row, int s) {
    uint8_t* d = ring + s * pitch;
    ptx::mbar_arrive_expect_tx(&full[s], bytes);
    if (!dbg_ok(row < rows && s < stages && stages <= kNormStages && stages * pitch <= kNormRingBytes &&
                    ((reinterpret_cast<uintptr_t>(row_ptr(p.dy, p.dy_dt, row, p.dys)) |
                      reinterpret_cast<uintptr_t>(row_ptr(p.h, p.h_dt, row, p.hs)) |
                      reinterpret_cast<uintptr_t>(has_res ? row_ptr(p.dres, p.dr_dt, row, p.drs) : nullptr) |
                      bd | bh | bs) & 15) == 0, p.status))
      return;                              // the wait for it runs out
    ptx::bulk_load(d, row_ptr(p.dy, p.dy_dt, row, p.dys), bd, &full[s]);
    ptx::bulk_load(d + bd, row_ptr(p.h, p.h_dt, row, p.hs), bh, &full[s]);
    if (has_res) ptx::bulk_load(d + bd + bh, row_ptr(p.dres, p.dr_dt, row, p.drs), bs, &full[s]);
  };
  if (t == 0) {
    for (int s = 0; s < stages; ++s) ptx::mbar_init(&full[s], 1);
    ptx::fence_mbar_init();
  }
  __syncthreads();
  if (t == 0)
    for (int s = 0; s < stages; ++s)
      if (p.inject && blockIdx.x == 0 && s == 0) ptx::mbar_arrive_expect_tx(&full[0], bytes);   // testing hook
      else if (blockIdx.x + static_cast<int64_t>(s) * step < rows) fetch(blockIdx.x + s * step, s);
  float2 acc[NV][4], g[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float v[8];
    load_gain(v, p.gain, p.g_dt, (i * tpr + t) * 8, p.cols, true);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      g[i][j] = make_float2(v[2 * j], v[2 * j + 1]);
      acc[i][j] = make_float2(0.f, 0.f);
    }
  }
  int s = 0, par = 0;
  uint32_t phase = 0;
  for (int64_t row = blockIdx.x; row < rows; row += step) {
    if (!ring_wait(&full[s], phase, p.status, p.timeout_ns)) {
      if (t == 0) ring_drain(full, stages, s, phase, (rows - 1 - row) / step + 1, p.status, p.timeout_ns);
      break;
    }
    const uint8_t* d = ring + s * pitch;
    Chunk<WIDE> cd[NV], ch[NV], cs[NV];
    float2 ss2 = make_float2(0.f, 0.f), dot2 = ss2;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * tpr + t) * 8;
      if (col >= p.cols) continue;
      load_chunk<WIDE>(cd[i], d, p.dy_dt, col, p.cols, true);
      load_chunk<WIDE>(ch[i], d + bd, p.h_dt, col, p.cols, true);
      if (has_res) load_chunk<WIDE>(cs[i], d + bd + bh, p.dr_dt, col, p.cols, true);
      float2 dv[4], h[4];
      to_float2<WIDE>(cd[i], p.dy_dt, dv);
      to_float2<WIDE>(ch[i], p.h_dt, h);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ss2 = ptx::fma2(h[j], h[j], ss2);
        dot2 = ptx::fma2(ptx::mul2(dv[j], g[i][j]), h[j], dot2);
      }
    }
    float ss = ss2.x + ss2.y, dot = dot2.x + dot2.y;
    row_reduce2(ss, dot, tpr, s_a[par], s_b[par]);
    const int64_t next = row + static_cast<int64_t>(stages) * step;
    if (t == 0 && next < rows) fetch(next, s);
    par ^= 1;
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
    const float rstd = rsqrtf(fmaf(ss, p.inv_cols, p.eps));
    const float m = -rstd * rstd * (dot * rstd * p.inv_cols);
    const float2 r2 = make_float2(rstd, rstd), m2 = make_float2(m, m);
    char* out = row_ptr(p.dh, p.dh_dt, row, p.dhs);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * tpr + t) * 8;
      if (col >= p.cols) continue;
      float2 dv[4], h[4], o[4];
      to_float2<WIDE>(cd[i], p.dy_dt, dv);
      to_float2<WIDE>(ch[i], p.h_dt, h);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = make_float2(0.f, 0.f);
      if (has_res) to_float2<WIDE>(cs[i], p.dr_dt, o);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][j] = ptx::fma2(ptx::mul2(dv[j], h[j]), r2, acc[i][j]);
        // rstd gain dy - rstd u mean + dres, u = h rstd
        o[j] = ptx::fma2(m2, h[j], ptx::fma2(r2, ptx::mul2(dv[j], g[i][j]), o[j]));
        v[2 * j] = o[j].x;
        v[2 * j + 1] = o[j].y;
      }
      store_chunk(out, p.dh_dt, col, p.cols, true, v);
    }
  }
  if (p.part) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * tpr + t) * 8;
      if (col >= p.cols) continue;
      const float v[8] = {acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y,
                          acc[i][2].x, acc[i][2].y, acc[i][3].x, acc[i][3].y};
      store_chunk(p.part + static_cast<int64_t>(blockIdx.x) * p.cols, kDtF32, col, p.cols, true, v);
    }
  }
}

// dgain[c] = sum over slots of part[slot][c], slots in a fixed order.
__global__ void __launch_bounds__(256) rmsnorm_dgain_kernel(const float* part, int slots, int cols,
                                                            float* dgain) {
  __shared__ float s[8][32];
  ptx::wait_dependency();
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
  const bool wide = p.x_dt != kDtBf16 || (p.r_dt != kDtNone && p.r_dt != kDtBf16);
  const int nv = p.rows <= 4 * sms && chunks <= 1024 ? 1 : wide && chunks <= 512 ? 2 : chunks <= 1024 ? 4 : 8;
  const int tpr = threads_per_row(p.cols, nv, 16);
  const int block = tpr > 32 ? tpr : 128;
  const int64_t grid = (p.rows + block / tpr - 1) / (block / tpr);
  const dim3 g(static_cast<unsigned>(grid));
  auto go = [&](auto nv_c) {
    constexpr int N = decltype(nv_c)::value;
    if (wide) rmsnorm_kernel<N, true><<<g, block, 0, s>>>(p, tpr);
    else rmsnorm_kernel<N, false><<<g, block, 0, s>>>(p, tpr);
  };
  if (nv == 1) go(std::integral_constant<int, 1>{});
  else if (nv == 2) go(std::integral_constant<int, 2>{});
  else if (nv == 4) go(std::integral_constant<int, 4>{});
  else go(std::integral_constant<int, 8>{});
  return cudaGetLastError();
}

namespace {

struct GradShape {
  int nv, tpr, block, grid;
  int stages;      // 0: rows loaded into registers
  int smem;
};

GradShape grad_shape(const NormGradParams& p, int sms) {
  GradShape g;
  const int chunks = (p.cols + 7) / 8;
  auto es = [](int dt) { return dt == kDtNone ? 0 : dt == kDtF32 ? 4 : 2; };
  g.stages = 0;
  g.smem = 0;
  // The ring: rows of whole 16-byte pieces, a block per row, two blocks on an
  // SM with at least two rows in flight each, and several rows per block.
  // 16384 x 4096 bf16 with a residual gradient: 80 us against 127 from registers.
  const int row = p.cols * (es(p.dy_dt) + es(p.h_dt) + es(p.dr_dt));
  const int pitch = (row + 127) / 128 * 128;
  if (p.vec && p.cols % 8 == 0 && chunks > 64 && chunks <= 1024 && 2 * pitch <= kNormRingBytes &&
      p.rows >= 8LL * sms) {
    g.nv = chunks <= 512 ? 2 : 4;
    g.tpr = g.block = ((chunks + g.nv - 1) / g.nv + 31) / 32 * 32;
    g.stages = std::min(kNormStages, kNormRingBytes / pitch);
    g.smem = g.stages * pitch;
    g.grid = 2 * sms;
    return g;
  }
  g.nv = p.rows <= 4 * sms && chunks <= 1024 ? 1 : chunks <= 512 ? 2 : chunks <= 1024 ? 4 : 8;
  g.tpr = threads_per_row(p.cols, g.nv, 8);
  g.block = g.tpr > 32 ? g.tpr : 128;
  const int per = g.block / g.tpr;
  const int64_t most = static_cast<int64_t>(sms) * std::max(1, 768 / g.block) * per;
  // rows a slot, then no more slots than that needs
  const int64_t turns = (p.rows + most - 1) / most;
  const int64_t slots = (p.rows + turns - 1) / turns;
  g.grid = static_cast<int>((slots + per - 1) / per);
  return g;
}

template <int NV, bool WIDE>
cudaError_t ring_launch(NormGradParams p, const GradShape& g, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(rmsnorm_grad_ring_kernel<NV, WIDE>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kNormRingBytes);
  if (e != cudaSuccess) return e;
  p.inject = take_injected_stall(kInjectGemm);
  rmsnorm_grad_ring_kernel<NV, WIDE><<<g.grid, g.block, g.smem, s>>>(p, g.stages);
  return cudaGetLastError();
}

}  // namespace

int norm_grad_slots(const NormGradParams& p, int sms) {
  const GradShape g = grad_shape(p, sms);
  return g.grid * (g.block / g.tpr);
}

cudaError_t launch_norm_grad(const NormGradParams& p, int sms, cudaStream_t s) {
  const GradShape g = grad_shape(p, sms);
  const bool wide = p.dy_dt != kDtBf16 || p.h_dt != kDtBf16 || (p.dr_dt != kDtNone && p.dr_dt != kDtBf16);
  if (g.stages) {
    if (g.nv == 2) return wide ? ring_launch<2, true>(p, g, s) : ring_launch<2, false>(p, g, s);
    return wide ? ring_launch<4, true>(p, g, s) : ring_launch<4, false>(p, g, s);
  }
  auto go = [&](auto nv_c) {
    constexpr int N = decltype(nv_c)::value;
    if (wide) rmsnorm_grad_kernel<N, true><<<g.grid, g.block, 0, s>>>(p, g.tpr);
    else rmsnorm_grad_kernel<N, false><<<g.grid, g.block, 0, s>>>(p, g.tpr);
  };
  if (g.nv == 1) go(std::integral_constant<int, 1>{});
  else if (g.nv == 2) go(std::integral_constant<int, 2>{});
  else if (g.nv == 4) go(std::integral_constant<int, 4>{});
  else go(std::integral_constant<int, 8>{});
  return cudaGetLastError();
}

cudaError_t launch_norm_dgain(const float* part, int slots, int cols, float* dgain, cudaStream_t s) {
  return launch_after(rmsnorm_dgain_kernel, (cols + 31) / 32, 256, 0, true, s, part, slots, cols, dgain);
}

}  // namespace muon
