// The experts' products over a routing (definitions at muon_experts_forward).
//
// Rows are (token, slot) pairs in expert order.  Each product is a grouped
// GEMM with the weights on the tensor cores' M side and the rows on the N
// side: N is any multiple of 32 up to 256, so an expert's rows are cut into
// equal tiles with at most 31 columns too many in each, whatever its count
// (a 128- or 256-row M tile would leave half a tile per expert idle).
//
//   up     D[f, r] = W_in[f, :] . x_r         gate and up rows interleaved by 8
//   down   D[h, r] = W_out[h, :] . act_r
//   dact   D[i, r] = W_out[:, i] . dout_r
//   dx     D[h, r] = W_in[:, h] . dgu_r
//   dw_in  D[f, h] = sum_r dgu[r, f] x[r, h]        K = the expert's rows
//   dw_out D[h, i] = sum_r dout[r, h] (w a)[r, i]
//
// One CTA pair (a cluster of two) per tile of 256 (M) x N: tcgen05.mma with
// cta_group::2, each CTA holding 128 rows of A, half of B's columns and 128
// rows of D, so 32 KB of operands feed each SM per 128 x 256 x 64 block.  Per CTA:
//   warp 0      TMA producer, a ring of six 32 KB stages (128-byte swizzle),
//               one copy per operand and stage: the copy engine's cost per
//               instruction shows (B in four boxes of 32 rows instead of one of
//               128: 1428 against 1207 us for 4093 tokens' up product over
//               8 x [28672, 4096]), which also rules out gathering the rows by
//               four in the copy, 32 instructions a stage.  Warps that gathered
//               16 bytes a thread straight into the stage took 0.5 us a stage
//               against 0.39 from a copy of the rows in expert order, more than
//               that copy costs;
//   warp 1      TMEM; in a pair's CTA 0 it issues the MMAs of both;
//   warps 2..9  epilogue, two sets of four (128 TMEM lanes each) that take
//               the accumulator's column slabs in turn.
// Two 256-column accumulators let the epilogue of a tile overlap the next
// tile's products.  Bound by the tensor cores where experts have hundreds of
// rows, by HBM (every weight read once) where they have a few.  4093 tokens
// through 2 of 8 x [14336, 4096]: up 1094 us, down 586 (1.76 and 1.64 PFLOP/s);
// 48 tokens through 8 of 256 x [768, 2048]: 225 us for 1.38 GB of weights, 0.90
// of the measured copy rate; 8192 tokens' gradient through 8 of 64 x
// [768, 2048]: dact 196, dx 298 (with x's copy beside it), dw_in 264, dw_out 155.
//
// The tile list follows from the offsets on the device: every CTA scans them
// (one warp, a few hundred cycles), so the host needs no counts.  Offsets are
// read as their running maximum clamped to [0, rows]: wrong ones give wrong
// values, not accesses out of range.  Every wait is bounded; on a timeout a
// status bit is set, copies in flight are awaited, TMEM is freed and the CTA
// returns.
//
// The gradient's buffers keep each expert's rows in a segment padded to 64
// rows with zeros: the weight gradients' K blocks then end with their
// expert's, and no row of another expert, nor anything unwritten, is ever
// multiplied.
#include <cuda_fp16.h>

#include <algorithm>

#include "block.h"
#include "block_ptx.cuh"

namespace muon {

namespace {

constexpr int BK = 64, UMMA_K = 16;
constexpr int kOpBytes = 128 * BK * 2;          // one CTA's A or B of a stage
constexpr int kStageBytes = 2 * kOpBytes;
constexpr int kMostStages = 6;
constexpr int kBarBytes = 256;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kThreads = 320;
// as for 480 threads: 136 registers, which leave room beside 10 warps for a
// block of the row copy (two warps in each quarter of the SM)
constexpr int kBoundThreads = 480;
constexpr uint32_t kTmemCols = 512;
constexpr unsigned kFull = 0xffffffffu;
// least exponent of a piece of rows: its factors both ways are normal numbers
constexpr uint32_t kExpLeast = 15;

constexpr bool is_dw(int kind) { return kind == kExDwIn || kind == kExDwOut; }
constexpr bool a_mn(int kind) { return kind >= kExDact; }   // A read MN-major

// epilogue staging per set
constexpr int set_bytes(int kind) {
  return is_dw(kind) ? 16 * 1024 : kind == kExDact ? 25 * 1024 : 12 * 1024;
}
int gemm_smem(int kind, int stages, int experts) {
  return stages * kStageBytes + 2 * set_bytes(kind) + kBarBytes + 3 * (experts + 1) * 4 + 1024;
}

// First row of every expert in the plan (off), in the padded numbering (poff)
// and its number of row tiles (tt, running).
struct Scan {
  int *off, *poff, *tt;    // [experts + 1]
};

__device__ __forceinline__ int round_up(int v, int to) { return (v + to - 1) / to * to; }

// All threads of the block: offsets into s.off, clamped; then, after a barrier,
// one warp scans.
__device__ __forceinline__ void fetch_offsets(const Scan& s, const int32_t* offsets, int experts,
                                              int64_t rows) {
  for (int e = threadIdx.x; e <= experts; e += blockDim.x)
    s.off[e] = max(0, static_cast<int>(min(static_cast<int64_t>(offsets[e]), rows)));
}

__device__ __forceinline__ void scan_offsets(const Scan& s, int experts, int pad, bool tile_pads, int lane) {
  int top = 0, pbase = 0, tbase = 0;
  for (int eb = 0; eb <= experts; eb += 32) {
    const int e = eb + lane;
    int v = e <= experts ? s.off[e] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kFull, v, o);
      if (lane >= o) v = max(v, u);
    }
    v = max(v, top);
    if (e <= experts) s.off[e] = v;
    top = __shfl_sync(kFull, v, 31);
  }
  __syncwarp();
  for (int eb = 0; eb < experts; eb += 32) {
    const int e = eb + lane;
    const int cnt = e < experts ? s.off[e + 1] - s.off[e] : 0;
    const int pc = round_up(cnt, pad);
    const int nt = ((tile_pads ? pc : cnt) + kExNTile - 1) / kExNTile;
    int a = pc, b = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kFull, a, o), w = __shfl_up_sync(kFull, b, o);
      if (lane >= o) {
        a += u;
        b += w;
      }
    }
    if (e < experts) {
      s.poff[e] = pbase + a - pc;
      s.tt[e] = tbase + b - nt;
    }
    pbase += __shfl_sync(kFull, a, 31);
    tbase += __shfl_sync(kFull, b, 31);
  }
  if (lane == 0) {
    s.poff[experts] = pbase;
    s.tt[experts] = tbase;
  }
}

// Largest e with v[e] <= x, for a non-decreasing v (empty experts skipped).
__device__ __forceinline__ int find(const int* v, int experts, int x) {
  int lo = 0, hi = experts - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (v[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

struct Tile {
  int e, m, n;          // expert, M tile, N tile (dw)
  int prow, urow;       // first row: padded and plan numbering
  int rows;             // rows to write
  int valid;            // rows of the plan among them
  int cols;             // MMA N, a multiple of 32
  int kb;               // K blocks
};

// Row tiles in groups of 8 per expert, M tiles outer and the group's row
// tiles inner: the pairs running at one time share a few weight panels and a
// few row panels, so that each comes from HBM once.
constexpr int kRowGroup = 8;

template <int KIND>
__device__ __forceinline__ Tile decode(const ExGemmParams& p, const Scan& s, int tile) {
  Tile t;
  if (is_dw(KIND)) {
    const int per = p.m_tiles * p.n_tiles;
    t.e = tile / per;
    const int r = tile - t.e * per;
    t.m = r / p.n_tiles;
    t.n = r - t.m * p.n_tiles;
    t.prow = s.poff[t.e];
    t.urow = s.off[t.e];
    t.rows = t.valid = 0;
    t.cols = kExNTile;
    t.kb = (s.poff[t.e + 1] - t.prow) / kExSeg;
    return t;
  }
  // the expert whose tiles [tt[e], tt[e + 1]) * m_tiles hold this one
  t.e = find(s.tt, p.experts, tile / p.m_tiles);
  const int nt = s.tt[t.e + 1] - s.tt[t.e];
  int local = tile - s.tt[t.e] * p.m_tiles;
  const int span = kRowGroup * p.m_tiles;
  const int g = local / span;
  local -= g * span;
  const int ge = min(kRowGroup, nt - g * kRowGroup);
  t.m = local / ge;
  const int j = g * kRowGroup + local - t.m * ge;
  const int cnt = s.off[t.e + 1] - s.off[t.e];
  const int all = KIND == kExDact ? round_up(cnt, p.pad) : cnt;
  const int size = round_up((all + nt - 1) / nt, 32);
  t.prow = s.poff[t.e] + j * size;
  t.urow = s.off[t.e] + j * size;
  t.rows = max(0, min(size, all - j * size));
  t.valid = max(0, min(size, cnt - j * size));
  t.cols = max(32, round_up(t.rows, 32));
  t.n = 0;
  t.kb = p.kb;
  return t;
}

// Debug builds: the tile's indices, and the rows that its copies and stores touch.
template <int KIND>
__device__ __forceinline__ bool tile_in_range(const ExGemmParams& p, const Tile& t) {
  const bool place = t.e >= 0 && t.e < p.experts && t.m >= 0 && t.m < p.m_tiles && t.prow >= 0 && t.kb >= 0;
  if (is_dw(KIND)) return place && t.n >= 0 && t.n < p.n_tiles && t.prow + static_cast<int64_t>(t.kb) * BK <= p.prows;
  return place && t.urow >= 0 && t.valid >= 0 && t.valid <= t.rows && t.rows <= t.cols && t.cols <= kExNTile &&
         t.cols % 32 == 0 && t.prow + static_cast<int64_t>(t.rows) <= p.prows &&
         t.urow + static_cast<int64_t>(t.valid) <= p.rows;
}

// A warp's tiles in order, decoded 32 at a time, one by each lane: decoding (a
// search of the offsets and four divisions, about 1200 cycles) once per tile in
// the copies' and the MMAs' threads cost a fifth of a tile of 12 K blocks.
template <int KIND>
struct Feed {
  Tile mine;
  // tile `it` of this pair; every lane calls it with the same `it`, in order
  __device__ __forceinline__ Tile get(const ExGemmParams& p, const Scan& s, int tiles, int tile0, int tstep,
                                      int it, int lane) {
    if ((it & 31) == 0) {
      const int64_t tile = tile0 + static_cast<int64_t>(it + lane) * tstep;
      if (tile < tiles) mine = decode<KIND>(p, s, static_cast<int>(tile));
    }
    Tile t;
    const int from = it & 31;
    t.e = __shfl_sync(kFull, mine.e, from);
    t.m = __shfl_sync(kFull, mine.m, from);
    t.n = __shfl_sync(kFull, mine.n, from);
    t.prow = __shfl_sync(kFull, mine.prow, from);
    t.urow = __shfl_sync(kFull, mine.urow, from);
    t.rows = __shfl_sync(kFull, mine.rows, from);
    t.valid = __shfl_sync(kFull, mine.valid, from);
    t.cols = __shfl_sync(kFull, mine.cols, from);
    t.kb = __shfl_sync(kFull, mine.kb, from);
    return t;
  }
};

// Waits are suspended in the hardware (up to 100 us at a time), not polled.
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                             unsigned* status, unsigned long long timeout_ns,
                                             bool honour_abort) {
  constexpr uint32_t kSuspendNs = 100000;
  const uint32_t addr = ptx::smem_u32(bar);
  if (ptx::mbar_try_wait_for(addr, parity, kSuspendNs)) return true;
  const uint64_t t0 = ptx::globaltimer();
  for (;;) {
    if (ptx::mbar_try_wait_for(addr, parity, kSuspendNs)) return true;
    if (honour_abort && *abort_flag) return false;
    if (ptx::globaltimer() - t0 > timeout_ns) {
      atomicOr(status, kDevTimeout);
      *abort_flag = 1;
      return false;
    }
  }
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float lo_of(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_of(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ float f(uint32_t v) { return __uint_as_float(v); }
// 1 / (1 + exp(-g)) by the approximate 2^x and 1 / x, each within 2 units of
// the last place of fp32; results are rounded to bf16.
__device__ __forceinline__ float sigmoid(float g) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}
__device__ __forceinline__ float2 sigmoid2(float2 g) { return make_float2(sigmoid(g.x), sigmoid(g.y)); }
__device__ __forceinline__ float2 f2(uint32_t lo, uint32_t hi) { return make_float2(f(lo), f(hi)); }
__device__ __forceinline__ float2 f2(uint32_t pair) { return make_float2(lo_of(pair), hi_of(pair)); }
__device__ __forceinline__ uint32_t pack(float2 v) { return pack(v.x, v.y); }
__device__ __forceinline__ uint32_t pack_half(float2 v) {
  const __half2 h = __float22half2_rn(v);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 of_half(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }

// 8 bf16 at p[0..8), of which the first n exist.
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* p, int n, bool vec) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (n <= 0) return v;
  if (vec && n >= 8) return *reinterpret_cast<const uint4*>(p);
  const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = j < n ? q[j] : 0u;
  v.x = w[0] | (w[1] << 16);
  v.y = w[2] | (w[3] << 16);
  v.z = w[4] | (w[5] << 16);
  v.w = w[6] | (w[7] << 16);
  return v;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const uint4& v, int n, bool vec) {
  if (n <= 0) return;
  if (vec && n >= 8) {
    *reinterpret_cast<uint4*>(p) = v;
    return;
  }
  uint16_t* q = reinterpret_cast<uint16_t*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) q[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
}

// Staging of 16-byte chunks, rows of `pitch` bytes, chunk index XOR row % 8:
// a column of eight rows and a row of eight chunks both touch all banks.
__device__ __forceinline__ uint32_t staged(uint32_t base, int row, int chunk, int pitch) {
  return base + row * pitch + ((chunk ^ (row & 7)) << 4);
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// What one warp of an epilogue set works on.
struct EpiWarp {
  uint32_t taddr;     // accumulator, this warp's 32 lanes
  uint32_t stg;       // the set's staging
  int set, q4, lane, tid;   // tid: 0..127 within the set
  int m0;             // first M row of this CTA
  __device__ void bar() const { ptx::named_bar(2 + set, 128); }
};

// Where a thread's 16-byte chunk of staged rows goes: rows `pitch` elements
// apart from `at`, all 8 columns (full) or the first n of them.  The epilogues
// are bound by instruction issue (two sets of four warps on an SM), so what a
// tile fixes is worked out once a tile and the common case is a bare store.
struct Out {
  __nv_bfloat16* at;
  int64_t pitch;
  int n;
  bool full;
  __device__ Out(__nv_bfloat16* base, int64_t row, int64_t pitch_, int col, int limit, bool vec)
      : at(base + row * pitch_ + col), pitch(pitch_), n(limit - col), full(vec && limit - col >= 8) {}
  __device__ __forceinline__ void put(int row, uint32_t staged_at) const {
    const uint4 v = lds16(staged_at);
    if (full) *reinterpret_cast<uint4*>(at + row * pitch) = v;
    else store8(at + row * pitch, v, n, false);
  }
};

// gate rows and up rows sit 8 lanes apart, so one thread holds a pair
__device__ __forceinline__ void epi_up(const ExGemmParams& p, const Tile& t, const EpiWarp& w) {
  const int f0 = w.m0 >> 1;      // first feature: half of this CTA's 128 rows are gates
  const int orow = w.tid >> 3, chunk = w.tid & 7, ft = f0 + chunk * 8;
  const Out act(p.act, t.prow + orow, p.ap, ft, p.ip, true);
  const Out gate(p.gu, t.urow + orow, 2 * p.inner, ft, p.inner, p.gu_vec != 0);
  const Out up(p.gu + p.inner, t.urow + orow, 2 * p.inner, ft, p.inner, p.gu_vec != 0);
  const uint32_t in0 = staged(w.stg, w.lane, w.q4 * 2, 128), in1 = staged(w.stg, w.lane, w.q4 * 2 + 1, 128);
  const uint32_t out = staged(w.stg, orow, chunk, 128);     // row + 16 keeps row % 8
  for (int c0 = w.set * 32; c0 < t.rows; c0 += 64) {
    uint32_t r[2][16];
    ptx::tmem_ld_16x256b_x4(w.taddr + c0, r[0]);
    ptx::tmem_ld_16x256b_x4(w.taddr + (16u << 16) + c0, r[1]);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint32_t a[4], g[4], u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 gv = f2(r[b][4 * i], r[b][4 * i + 1]), uv = f2(r[b][4 * i + 2], r[b][4 * i + 3]);
        a[i] = pack(ptx::mul2(ptx::mul2(gv, sigmoid2(gv)), uv));
        g[i] = pack(gv);
        u[i] = pack(uv);
      }
      const uint32_t in = b ? in1 : in0;
      ptx::stmatrix_x4_trans(in, a);
      if (p.gu) {
        ptx::stmatrix_x4_trans(in + 4096, g);
        ptx::stmatrix_x4_trans(in + 8192, u);
      }
    }
    w.bar();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int row = c0 + 16 * k;
      if (row + orow >= t.rows || act.n <= 0) continue;
      act.put(row, out + 2048 * k);
      if (p.gu) {
        gate.put(row, out + 4096 + 2048 * k);
        up.put(row, out + 8192 + 2048 * k);
      }
    }
    w.bar();
  }
}

// Rows for the sum over slots, as 16-bit floats (IEEE half) with one exponent
// per row and 32 features (a warp's lanes): q = v * 2^(14 - e), e the exponent of
// the piece's largest finite value; infinities and NaN stay what and where they
// are.  A value keeps 11 bits while it is above 2^-28 of that largest one (below,
// its error is 2^-39 of it): a term errs by at most 2^-11 of itself, an eighth of
// what the bf16 operand behind it and the bf16 result add, whatever its neighbours
// hold.  (15-bit integers, uniform in a piece, gave a feature beside one 1000
// times larger an error of 2.6 %; bf16 rows would add as much as the result's
// rounding.)  Half of fp32's bytes are written and read (16384 tokens over 256 x
// [768, 2048], product and sum: 398 + 167 us with fp32 rows, 378 + 91 with 16 bits
// when they were compared; 327 + 93 now).
__device__ __forceinline__ void epi_rows(const ExGemmParams& p, const Tile& t, const EpiWarp& w) {
  const int orow = w.tid >> 4, chunk = w.tid & 15, h = w.m0 + chunk * 8;
  __half* const y = p.y + static_cast<int64_t>(t.urow + orow) * p.yp + h;
  uint8_t* const ex = p.yexp + static_cast<int64_t>(t.urow + w.lane) * p.yep + (w.m0 >> 5) + w.q4;
  const bool mine = h < p.yp;
  const uint32_t out = staged(w.stg, orow, chunk, 256);     // row + 8 keeps row % 8
  for (int c0 = w.set * 32; c0 < t.rows; c0 += 64) {
    uint32_t r[2][16];
    ptx::tmem_ld_16x256b_x4(w.taddr + c0, r[0]);
    ptx::tmem_ld_16x256b_x4(w.taddr + (16u << 16) + c0, r[1]);
    ptx::tmem_ld_wait();
    // rows 8 i + 2 (lane % 4) (low half) and the next (high half): upper 16 bits
    // of the magnitudes, largest over this thread's 4 features, then the warp's 32
    uint32_t m[4];
    auto largest = [&](bool only_finite) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] = 0;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t v = __byte_perm(r[b][4 * i + 2 * q], r[b][4 * i + 2 * q + 1], 0x7632) & 0x7fff7fffu;
            if (only_finite) v &= ~__vcmpgeu2(v, 0x7f807f80u);
            m[i] = __vmaxu2(m[i], v);
          }
      }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = __vmaxu2(m[i], __shfl_xor_sync(kFull, m[i], o));
    };
    largest(false);
    if (__any_sync(kFull, __vmaxu2(__vmaxu2(__vmaxu2(m[0], m[1]), __vmaxu2(m[2], m[3])), 0x7f7f7f7fu) != 0x7f7f7f7fu))
      largest(true);
    uint32_t e32 = 0;      // exponent of row c0 + lane, from a lane that holds its i and pair
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = __shfl_sync(kFull, m[i], (w.lane >> 1) & 3);
      if ((w.lane >> 3) == i) e32 = (w.lane & 1) ? v >> 23 : (v >> 7) & 0xffu;
    }
    if (c0 + w.lane < t.rows && w.m0 < p.m) ex[c0 * p.yep] = static_cast<uint8_t>(max(e32, kExpLeast));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 s;
      s.x = f((268u - max((m[i] >> 7) & 0xffu, kExpLeast)) << 23);
      s.y = f((268u - max(m[i] >> 23, kExpLeast)) << 23);
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t* v = &r[b][4 * i + 2 * q];
          v[0] = pack_half(ptx::mul2(f2(v[0], v[1]), s));
        }
    }
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t v[4] = {r[b][2 * q], r[b][4 + 2 * q], r[b][8 + 2 * q], r[b][12 + 2 * q]};
        ptx::stmatrix_x4_trans(staged(w.stg, w.lane, w.q4 * 4 + b * 2 + q, 256), v);
      }
    w.bar();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = c0 + 8 * k;
      if (row + orow < t.rows && mine) *reinterpret_cast<uint4*>(y + row * p.yp) = lds16(out + 2048 * k);
    }
    w.bar();
  }
}

// The tile's row weights into the set's staging, past the slabs.
constexpr int kWeightOff = 24 * 1024;
__device__ __forceinline__ void fetch_weights(const ExGemmParams& p, const Tile& t, const EpiWarp& w) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int row = w.tid + 128 * k;
    const float v = row < t.valid ? p.wr[t.prow + row] : 0.f;
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(w.stg + kWeightOff + row * 4), "f"(v) : "memory");
  }
}

// Gate and up rows of a slab of 32 rows, into registers: asked for a slab (and
// a tile's first before its products are done) early, as their latency is a
// slab's arithmetic.
struct GateUp {
  uint4 v[8];     // rows tid / 16 + 8 k of the gates, then of the ups
};
__device__ __forceinline__ void fetch_gu(const ExGemmParams& p, const Tile& t, const EpiWarp& w, int c0,
                                         GateUp& in) {
  const int row = c0 + (w.tid >> 4), ft = w.m0 + (w.tid & 15) * 8, n = p.inner - ft;
  const int64_t pitch = 2 * p.inner;
  const __nv_bfloat16* q = p.gu + (t.urow + row) * pitch + ft;
  if (p.gu_vec && n >= 8) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      in.v[k] = in.v[k + 4] = make_uint4(0u, 0u, 0u, 0u);
      if (row + 8 * k < t.valid) {
        in.v[k] = *reinterpret_cast<const uint4*>(q + 8 * k * pitch);
        in.v[k + 4] = *reinterpret_cast<const uint4*>(q + 8 * k * pitch + p.inner);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      in.v[k] = load8(q + 8 * (k & 3) * pitch + (k >> 2) * p.inner, row + 8 * (k & 3) < t.valid ? n : 0, false);
  }
}

// da -> dgu, w a and this warp's 32 features' part of <da, a>; 32 rows at a time
__device__ __forceinline__ void epi_dact(const ExGemmParams& p, const Tile& t, const EpiWarp& w, GateUp& in) {
  const int orow = w.tid >> 4, chunk = w.tid & 15, ft = w.m0 + chunk * 8;
  constexpr uint32_t kUp = 8192, kAct = 16384;
  const Out dg_out(p.dgu, t.prow + orow, p.gp, ft, p.ip, true);
  const Out du_out(p.dgu + p.ip, t.prow + orow, p.gp, ft, p.ip, true);
  const Out wa_out(p.act, t.prow + orow, p.ap, ft, p.ip, true);
  const uint32_t own = staged(w.stg, orow, chunk, 256);     // row + 8 keeps row % 8
  float* const part = p.part + ((w.m0 >> 5) + w.q4) * p.rows + t.urow + 2 * (w.lane & 3);
  const bool parts = w.lane < 4 && w.m0 < p.m;
  // ldmatrix / stmatrix: matrix 2 i + c is rows 8 i.. of 8 features, chunk c of a 16-lane block
  const int lr = (w.lane >> 4) * 8 + (w.lane & 7), lc = w.q4 * 4 + ((w.lane >> 3) & 1);
  const uint32_t mat[2] = {staged(w.stg, lr, lc, 256), staged(w.stg, lr, lc + 2, 256)};
  for (int c0 = w.set * 32; c0 < t.rows; c0 += 64) {
#pragma unroll
    for (int k = 0; k < 8; ++k) sts16(own + (k >> 2) * kUp + (k & 3) * 2048, in.v[k]);
    if (c0 + 64 < t.rows) fetch_gu(p, t, w, c0 + 64, in);
    w.bar();
#pragma unroll
    for (int s = 0; s < 2; ++s) {       // 16 rows
      const int cs = c0 + 16 * s;
      float2 wt[2], dot[2];             // rows cs + 8 i + 2 (lane % 4) and the next
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                     : "=f"(wt[i].x), "=f"(wt[i].y)
                     : "r"(w.stg + kWeightOff + (cs + 8 * i + 2 * (w.lane & 3)) * 4)
                     : "memory");
        dot[i] = make_float2(0.f, 0.f);
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t r[8], g[4], u[4], a[4];
        ptx::tmem_ld_16x256b_x2(w.taddr + (static_cast<uint32_t>(b * 16) << 16) + cs, r);
        const uint32_t at = mat[b] + s * 4096;
        ptx::ldmatrix_x4_trans(at, g);
        ptx::ldmatrix_x4_trans(at + kUp, u);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float2 gv = f2(g[2 * i + c]), uv = f2(u[2 * i + c]);
            const float2 da = f2(r[4 * i + 2 * c], r[4 * i + 2 * c + 1]);
            const float2 sg = sigmoid2(gv);
            const float2 sl = ptx::mul2(gv, sg), act = ptx::mul2(sl, uv), wd = ptx::mul2(wt[i], da);
            dot[i] = ptx::fma2(da, act, dot[i]);
            // silu' = s (1 + g - g s) = s + sl - sl s
            const float2 slope = ptx::fma2(make_float2(-sl.x, -sl.y), sg, ptx::add2(sl, sg));
            g[2 * i + c] = pack(ptx::mul2(ptx::mul2(wd, uv), slope));
            u[2 * i + c] = pack(ptx::mul2(wd, sl));
            a[2 * i + c] = pack(ptx::mul2(wt[i], act));
          }
        // a warp reads and writes its own four chunks only
        ptx::stmatrix_x4_trans(at, g);
        ptx::stmatrix_x4_trans(at + kUp, u);
        ptx::stmatrix_x4_trans(at + kAct, a);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          dot[i].x += __shfl_xor_sync(kFull, dot[i].x, o);
          dot[i].y += __shfl_xor_sync(kFull, dot[i].y, o);
        }
        const int row = cs + 8 * i + 2 * (w.lane & 3);
        if (parts && row < t.valid) part[cs + 8 * i] = dot[i].x;
        if (parts && row + 1 < t.valid) part[cs + 8 * i + 1] = dot[i].y;
      }
    }
    w.bar();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = c0 + 8 * k;
      if (row + orow >= t.rows || dg_out.n <= 0) continue;
      dg_out.put(row, own + k * 2048);
      du_out.put(row, own + kUp + k * 2048);
      wa_out.put(row, own + kAct + k * 2048);
    }
    w.bar();
  }
}

// Weight gradients: lane = row, 128 bytes of columns at a time.
template <int KIND>
__device__ __forceinline__ void epi_dw(const ExGemmParams& p, const Tile& t, const EpiWarp& w) {
  const bool f32 = p.dw_dt == kDtF32;
  const int slab = f32 ? 32 : 64, per = f32 ? 4 : 8;   // columns per slab and 16-byte chunk
  const int n0 = t.n * kExNTile;
  const int row = w.q4 * 32 + w.lane;
  for (int c0 = w.set * slab; c0 < kExNTile && n0 + c0 < p.n; c0 += 2 * slab) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h && f32) break;
      uint32_t r[32];
      if (t.kb > 0) {
        ptx::tmem_ld_32x32b_x32(w.taddr + c0 + 32 * h, r);
        ptx::tmem_ld_wait();
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) r[j] = 0u;
      }
      if (f32) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          sts16(staged(w.stg, row, c, 128), make_uint4(r[4 * c], r[4 * c + 1], r[4 * c + 2], r[4 * c + 3]));
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          sts16(staged(w.stg, row, 4 * h + c, 128),
                make_uint4(pack(f(r[8 * c]), f(r[8 * c + 1])), pack(f(r[8 * c + 2]), f(r[8 * c + 3])),
                           pack(f(r[8 * c + 4]), f(r[8 * c + 5])), pack(f(r[8 * c + 6]), f(r[8 * c + 7]))));
      }
    }
    w.bar();
    const int chunk = w.tid & 7, col = n0 + c0 + chunk * per;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int rr = (w.tid >> 3) + 16 * k;
      int m = w.m0 + rr;
      bool ok = m < p.m;
      int64_t m_out = p.m;
      if (KIND == kExDwIn) {     // [2][ip] rows -> [2][inner]
        const int half = m >= p.ip;
        m -= half * p.ip;
        ok = ok && m < p.inner;
        m += half * p.inner;
        m_out = 2 * p.inner;
      }
      if (!ok || col >= p.n) continue;
      const uint4 v = lds16(staged(w.stg, rr, chunk, 128));
      const int64_t at = (t.e * m_out + m) * p.n + col;
      if (!dbg_ok(at + min(per, p.n - col) <= p.experts * m_out * p.n, p.status)) continue;
      if (!f32) {
        store8(static_cast<__nv_bfloat16*>(p.dw) + at, v, p.n - col, p.dw_vec != 0);
      } else {
        float* o = static_cast<float*>(p.dw) + at;
        if (p.dw_vec && p.n - col >= 4) {
          *reinterpret_cast<uint4*>(o) = v;
        } else {
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j < p.n - col) o[j] = f(u[j]);
        }
      }
    }
    w.bar();
  }
}

}  // namespace

template <int KIND, int PAIRS>
__global__ void __cluster_dims__(2 * PAIRS, 1, 1) __launch_bounds__(kBoundThreads, 1)
    ex_gemm_kernel(const __grid_constant__ ExGemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  const int kStages = p.stages;
  uint8_t* sStage = smem;
  uint8_t* sEpi = smem + kStages * kStageBytes;
  uint8_t* sBar = sEpi + 2 * set_bytes(KIND);
  uint64_t* full = reinterpret_cast<uint64_t*>(sBar);   // a pair's CTA 0 counts for both
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;     // [2] accumulator ready
  uint64_t* tempty = tfull + 2;          // [2] accumulator drained by the pair (its CTA 0's)
  uint64_t* mma_drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* s_ok = reinterpret_cast<volatile int*>(tmem_slot + 2);   // [2 sets][2]
  Scan scan;
  scan.off = reinterpret_cast<int*>(sBar + kBarBytes);
  scan.poff = scan.off + p.experts + 1;
  scan.tt = scan.poff + p.experts + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(ptx::cluster_ctarank());
  const int crank = rank & 1, pair = rank >> 1;      // place in the pair; pair of the cluster
  const int tile0 = static_cast<int>(blockIdx.x) / (2 * PAIRS), tstep = static_cast<int>(gridDim.x) / (2 * PAIRS);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], PAIRS);      // each pair's MMAs are done with it
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&tfull[b], 1);
      ptx::mbar_init(&tempty[b], 16);    // the epilogue warps of both CTAs
    }
    ptx::mbar_init(mma_drain, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&p.mapA);
    ptx::prefetch_tmap(&p.mapB);
    if (!is_dw(KIND)) ptx::prefetch_tmap(&p.mapB32);
  }
  if (warp == 1) ptx::tmem_alloc_pair(tmem_slot, kTmemCols);
  fetch_offsets(scan, p.offsets, p.experts, p.rows);
  __syncthreads();
  if (warp == 2) scan_offsets(scan, p.experts, p.pad, KIND == kExDact, lane);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();     // every CTA's barriers are initialised
  ptx::tc_fence_after();
  ptx::launch_dependents();
  if (!p.beside) ptx::wait_dependency();
  const uint32_t tmem = *tmem_slot;
  // tiles of the cluster: PAIRS M tiles and one column tile each
  const int tiles = is_dw(KIND) ? p.experts * p.m_tiles * p.n_tiles : scan.tt[p.experts] * p.m_tiles;
  auto m_first = [&](const Tile& t) { return (t.m * PAIRS + pair) * kExMTile + crank * 128; };

  if (warp == 0) {
    // ---- TMA producer (lane 0; the others hold tiles) -----------------------------------
    Feed<KIND> feed;
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    bool stop = false;
    const uint32_t full0 = ptx::mapa_shared(ptx::smem_u32(full), rank & ~1);
    for (int tile = tile0, it = 0; tile < tiles && !stop; tile += tstep, ++it) {
      const Tile t = feed.get(p, scan, tiles, tile0, tstep, it, lane);
      if (!dbg_ok(tile_in_range<KIND>(p, t), p.status)) break;      // consumers time out
      // B: 128 rows in boxes of 128 / PAIRS, one from each pair for all; for a
      // small tile one or two boxes of 32
      const int half = t.cols / 2, small = half > 64 ? 0 : (half + 31) / 32;
      const uint32_t bytes = 2 * (kOpBytes + (small ? small * 4096 : kOpBytes));
      const int m0 = m_first(t);
      const uint16_t mask = static_cast<uint16_t>(PAIRS == 2 ? 0x5 << crank : 0);
      for (int i = 0; lane == 0 && i < t.kb; ++i) {
        if (!wait_bounded(&empty[stage], phase ^ 1, abort_flag, p.status, p.timeout_ns, true)) {
          stop = true;
          break;
        }
        if (crank == 0) ptx::mbar_arrive_expect_tx(&full[stage], bytes);
        const uint32_t bar = full0 + stage * 8;
        uint8_t* a = sStage + stage * kStageBytes;
        uint8_t* b = a + kOpBytes;
        const int k = i * BK;
        if (KIND == kExUp) {
          // 8 features x (gate, up) x 8 groups: 128 rows
          ptx::tma_load_5d_pair(a, &p.mapA, bar, k, 0, 0, m0 >> 4, t.e);
        } else if (KIND == kExDown) {
          ptx::tma_load_3d_pair(a, &p.mapA, bar, k, m0, t.e);
        } else if (is_dw(KIND)) {
          ptx::tma_load_3d_pair(a, &p.mapA, bar, 0, t.prow + k, m0 / 64);
        } else if (p.a_whole) {
          ptx::tma_load_4d_pair(a, &p.mapA, bar, 0, k, m0 / 64, t.e);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            ptx::tma_load_3d_pair(a + h * 8192, &p.mapA, bar, m0 + 64 * h, k, t.e);
        }
        if (PAIRS == 1) {
          if (is_dw(KIND)) {
            ptx::tma_load_3d_pair(b, &p.mapB, bar, 0, t.prow + k, t.n * 4 + crank * 2);
          } else if (small == 0) {
            ptx::tma_load_2d_pair(b, &p.mapB, bar, k, t.prow + crank * half);
          } else {
            for (int h = 0; h < small; ++h)
              ptx::tma_load_2d_pair(b + h * 4096, &p.mapB32, bar, k, t.prow + crank * half + 32 * h);
          }
        } else if (is_dw(KIND)) {
          ptx::tma_load_3d_pair_mc(b + pair * 8192, &p.mapB, bar, 0, t.prow + k, t.n * 4 + crank * 2 + pair, mask);
        } else if (small == 0) {
          ptx::tma_load_2d_pair_mc(b + pair * 8192, &p.mapB, bar, k, t.prow + crank * half + 64 * pair, mask);
        } else if (pair < small) {
          ptx::tma_load_2d_pair_mc(b + pair * 4096, &p.mapB32, bar, k, t.prow + crank * half + 32 * pair, mask);
        }
        ++issued;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      stop = __shfl_sync(kFull, stop, 0);
    }
    // CTA 0: the last copies into both CTAs have landed before the pair exits
    if (crank == 0 && lane == 0)
      for (int j = issued > kStages ? issued - kStages : 0; j < issued; ++j)
        wait_bounded(&full[j % kStages], (j / kStages) & 1, abort_flag, p.status, p.timeout_ns, false);
    __syncwarp();
  } else if (warp == 1) {
    // ---- MMA issuer (a pair's CTA 0, lane 0; the others hold tiles) -------------------------------
    if (crank == 0) {
      Feed<KIND> feed;
      int stage = 0, acc = 0;
      uint32_t phase = 0;
      bool stop = false;
      const uint32_t s0 = ptx::smem_u32(sStage);
      const uint64_t desc_a = a_mn(KIND) ? ptx::sdesc_mnmajor_sw128(s0, 8192, 1024) : ptx::sdesc_kmajor_sw128(s0);
      const uint64_t desc_b = is_dw(KIND) ? ptx::sdesc_mnmajor_sw128(s0 + kOpBytes, 8192, 1024)
                                          : ptx::sdesc_kmajor_sw128(s0 + kOpBytes);
      const uint32_t a_lo = static_cast<uint32_t>(desc_a), b_lo = static_cast<uint32_t>(desc_b);
      const uint64_t a_hi = desc_a >> 32 << 32, b_hi = desc_b >> 32 << 32;
      if (p.inject && blockIdx.x == 0) {      // testing hook: nothing arrives there before the end
        if (lane == 0) stop = !wait_bounded(mma_drain, 0, abort_flag, p.status, p.timeout_ns, false);
        stop = __shfl_sync(kFull, stop, 0);
      }
      for (int tile = tile0, it = 0; tile < tiles && !stop; tile += tstep, ++it) {
        const Tile t = feed.get(p, scan, tiles, tile0, tstep, it, lane);
        if (t.kb == 0) continue;
        const uint32_t idesc = ptx::idesc_bf16_f32(kExMTile, t.cols) | (a_mn(KIND) ? 1u << 15 : 0u) |
                               (is_dw(KIND) ? 1u << 16 : 0u);
        const int buf = acc & 1;
        const uint32_t d = tmem + buf * 256;
        if (lane == 0) {
          stop = !wait_bounded(&tempty[buf], ((acc >> 1) & 1) ^ 1, abort_flag, p.status, p.timeout_ns, true);
          ptx::tc_fence_after();
          uint32_t acc_on = 0;      // the tile's first MMA overwrites
          for (int i = 0; i < t.kb && !stop; ++i) {
            if (!wait_bounded(&full[stage], phase, abort_flag, p.status, p.timeout_ns, true)) {
              stop = true;
              break;
            }
            ptx::tc_fence_after();
            // Addresses move in the descriptors' low word only (16-byte units),
            // so a K block costs this thread a handful of additions: built anew,
            // eight descriptors took longer than the MMAs they feed.
            const uint32_t at = stage * (kStageBytes >> 4);
#pragma unroll
            for (int k = 0; k < BK / UMMA_K; ++k) {
              // K-major: along the 128-byte row; MN-major: 16 rows (two 1024-byte atoms)
              const uint32_t da = a_lo + at + k * (a_mn(KIND) ? 2048 >> 4 : (UMMA_K * 2) >> 4);
              const uint32_t db = b_lo + at + k * (is_dw(KIND) ? 2048 >> 4 : (UMMA_K * 2) >> 4);
              ptx::umma_bf16_pair(d, a_hi | da, b_hi | db, idesc, acc_on);
              acc_on = 1;
            }
            ptx::umma_commit_pair(&empty[stage], PAIRS == 1 ? 0x3 : 0xf);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
          ptx::umma_commit_pair(&tfull[buf], static_cast<uint16_t>(0x3 << (2 * pair)));
        }
        ++acc;
        stop = __shfl_sync(kFull, stop, 0);
      }
      // no MMA may still run when TMEM is freed
      if (lane == 0) {
        ptx::umma_commit_pair(mma_drain, static_cast<uint16_t>(1 << rank));
        wait_bounded(mma_drain, 0, abort_flag, p.status, p.timeout_ns, false);
      }
    }
    __syncwarp();
  } else {
    // ---- epilogue --------------------------------------------------------------------------
    EpiWarp w;
    w.q4 = warp & 3;       // TMEM lane quadrant this warp may read
    w.set = (warp - 2) >> 2;
    w.lane = lane;
    w.tid = ((warp - 2) & 3) * 32 + lane;
    w.stg = ptx::smem_u32(sEpi + w.set * set_bytes(KIND));
    int acc = 0;
    Feed<KIND> feed;
    for (int tile = tile0, it = 0; tile < tiles; tile += tstep, ++it) {
      const Tile t = feed.get(p, scan, tiles, tile0, tstep, it, lane);
      if (!dbg_ok(tile_in_range<KIND>(p, t), p.status)) break;
      w.m0 = m_first(t);
      const int buf = acc & 1;
      w.taddr = tmem + buf * 256 + (static_cast<uint32_t>(w.q4 * 32) << 16);
      GateUp in;
      if (KIND == kExDact) {
        fetch_weights(p, t, w);
        if (w.set * 32 < t.rows) fetch_gu(p, t, w, w.set * 32, in);
      }
      if (t.kb > 0) {
        // One thread of the set waits and decides for all (they share a barrier,
        // which costs nothing while it holds them); the slot alternates with the
        // accumulator, so the next tile that waits has its barrier between two uses.
        if (w.tid == 0) {
          wait_bounded(&tfull[buf], (acc >> 1) & 1, abort_flag, p.status, p.timeout_ns, false);
          s_ok[2 * w.set + buf] = !*abort_flag;
        }
        w.bar();
        if (!s_ok[2 * w.set + buf]) break;
        ptx::tc_fence_after();
      }
      if (KIND == kExUp) epi_up(p, t, w);
      else if (KIND == kExDact) epi_dact(p, t, w, in);
      else if (is_dw(KIND)) epi_dw<KIND>(p, t, w);
      else epi_rows(p, t, w);
      if (t.kb > 0) {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster_relaxed(ptx::mapa_shared(ptx::smem_u32(&tempty[buf]), rank & ~1));
        ++acc;
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();     // no copy, MMA or arrival still aims at the partner
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc_pair(tmem, kTmemCols);
  if (p.beside) ptx::wait_dependency();      // this kernel's end is also that one's
}

// Copies the rows of x (or dout) into expert order: a warp reads a token's
// columns once, eight 16-byte loads a lane in flight and the next token's rows
// with them, and writes them to each of its rows.  HBM-bound: 65536 rows of 2048
// in 54 us (5.6 TB/s); 77 with a warp per row, which reads a token top_k times.
__global__ void __launch_bounds__(256, 5) ex_spread_kernel(const __grid_constant__ ExSpreadParams p) {
  extern __shared__ int s_scan[];
  Scan s;
  s.off = s_scan;
  s.poff = s.off + p.experts + 1;
  s.tt = s.poff + p.experts + 1;
  const int lane = threadIdx.x & 31;
  ptx::launch_dependents();
  fetch_offsets(s, p.offsets, p.experts, p.rows);
  __syncthreads();
  if (threadIdx.x < 32) scan_offsets(s, p.experts, p.pad, false, lane);
  __syncthreads();
  const int total = s.off[p.experts];
  const int step = gridDim.x * 8, first = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int begin = blockIdx.y * p.span, end = min(begin + p.span, static_cast<int>(p.hp));
  const int tokens = static_cast<int>(p.tokens), hidden = static_cast<int>(p.hidden);
  // row of this lane's slot of a token
  auto slot = [&](int64_t tok) {
    return tok < tokens && lane < p.top_k ? p.pos[tok * p.top_k + lane] : -1;
  };
  int next = slot(first);
  for (int64_t tok = first; tok < tokens; tok += step) {
    int row = next < total ? next : -1;
    next = slot(tok + step);
    if (p.pad > 1 && row >= 0) {
      const int e = find(s.off, p.experts, row);
      row += s.poff[e] - s.off[e];
    }
    if (!dbg_ok(row < p.prows, p.status)) row = -1;
    const unsigned live = __ballot_sync(kFull, row >= 0);
    if (!live) continue;
    const __nv_bfloat16* in = p.x + tok * p.xs;
    for (int cb = begin; cb < end; cb += 2048) {
      const int c0 = cb + lane * 8;
      uint4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = c0 + 256 * j;
        v[j] = load8(in + c, c < end ? min(hidden - c, 8) : 0, p.vec != 0);
      }
      for (unsigned m = live; m; m &= m - 1) {
        __nv_bfloat16* out = p.out + __shfl_sync(kFull, row, __ffs(m) - 1) * p.hp;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c0 + 256 * j < end) *reinterpret_cast<uint4*>(out + c0 + 256 * j) = v[j];
      }
    }
    if (p.wr && row >= 0 && begin == 0) p.wr[row] = p.weights[tok * p.top_k + lane];
  }
  // zeros after each expert's rows
  for (int i = first; p.pad > 1 && i < p.experts * p.pad; i += step) {
    const int e = i / p.pad, r = s.poff[e] + s.off[e + 1] - s.off[e] + i % p.pad;
    if (r >= s.poff[e + 1] || !dbg_ok(r < p.prows, p.status)) continue;
    for (int c = begin + lane * 8; c < end; c += 256)
      *reinterpret_cast<uint4*>(p.out + r * p.hp + c) = make_uint4(0u, 0u, 0u, 0u);
    if (p.wr && lane == 0 && begin == 0) p.wr[r] = 0.f;
  }
  if (p.beside) ptx::wait_dependency();      // this kernel's end is also that one's
}

// out[t] = sum over slots, in slot order, a block per token, eight columns a
// lane, SLOTS slots' loads in flight and the next token's rows with them;
// HBM-bound once the conversions are few (no branch per slot: a slot without a row
// reads row 0 and takes zeros): 16384 tokens of 8 slots of 2048 in 93 us, 6.3 TB/s.
template <int SLOTS>
__global__ void __launch_bounds__(256, 3) ex_combine_kernel(const __grid_constant__ ExCombineParams p) {
  const int lane = threadIdx.x & 31;
  const uint32_t tokens = static_cast<uint32_t>(p.tokens);      // below 2^31, as is its slots' number
  const int hidden = static_cast<int>(p.hidden);
  const int yp = static_cast<int>(p.yp), yep = static_cast<int>(p.yep);
  // this lane's slot of a token: its row, -1 for none, and weight
  auto slot = [&](uint32_t t, int32_t* row, float* w) {
    *row = -1;
    *w = 1.f;
    if (t >= tokens || lane >= p.top_k) return;
    *row = p.pos[t * p.top_k + lane];
    if (p.weights) *w = p.weights[t * p.top_k + lane];
  };
  ptx::launch_dependents();
  int32_t next_row;
  float next_w;
  slot(blockIdx.x, &next_row, &next_w);
  ptx::wait_dependency();
  for (uint32_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    const int32_t my_row = next_row < p.rows ? next_row : -1;
    const float my_w = my_row >= 0 ? next_w : 0.f;
    slot(t + gridDim.x, &next_row, &next_w);
    for (int c = threadIdx.x * 8; c - lane * 8 < hidden; c += blockDim.x * 8) {
      const int cr = min(c, static_cast<int>(p.yp) - 8);      // read column
      const unsigned live = __ballot_sync(kFull, my_row >= 0);
      float2 v[4] = {};
      for (int j0 = 0; j0 < p.top_k; j0 += SLOTS) {      // j0 + j < 32: top_k is at most 32
        uint4 y[SLOTS];
        uint32_t e[SLOTS];
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
          const int64_t r = max(__shfl_sync(kFull, my_row, j0 + j), 0);
          y[j] = *reinterpret_cast<const uint4*>(p.y + r * yp + cr);
          e[j] = p.yexp[r * yep + (cr >> 5)];
        }
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
          const float wj = __shfl_sync(kFull, my_w, j0 + j);
          const float w = wj * f((max(e[j], kExpLeast) - 14u) << 23);
          const float2 w2 = make_float2(w, w);
          if (!((live >> (j0 + j)) & 1u)) y[j] = make_uint4(0u, 0u, 0u, 0u);
          v[0] = ptx::fma2(w2, of_half(y[j].x), v[0]);
          v[1] = ptx::fma2(w2, of_half(y[j].y), v[1]);
          v[2] = ptx::fma2(w2, of_half(y[j].z), v[2]);
          v[3] = ptx::fma2(w2, of_half(y[j].w), v[3]);
        }
      }
      const uint4 o = make_uint4(pack(v[0].x, v[0].y), pack(v[1].x, v[1].y), pack(v[2].x, v[2].y),
                                 pack(v[3].x, v[3].y));
      store8(p.out + t * p.outs + c, o, hidden - c, p.vec != 0);
    }
  }
}

__global__ void __launch_bounds__(256) ex_dweights_kernel(const __grid_constant__ ExWeightParams p) {
  ptx::launch_dependents();
  ptx::wait_dependency();
  for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < p.rows; i += gridDim.x * 256LL) {
    const int32_t r = p.pos[i];
    float v = 0.f;
    if (r >= 0 && r < p.rows)
      for (int k = 0; k < p.parts; ++k) v += p.part[k * p.rows + r];
    p.dweights[i] = v;
  }
}

__global__ void __launch_bounds__(256)
    ex_repack_kernel(const __nv_bfloat16* in, int64_t mats, int64_t rows, int64_t cols, __nv_bfloat16* out,
                     int64_t rows_p, int64_t cols_p) {
  const int lane = threadIdx.x & 31;
  for (int64_t r = blockIdx.x * 8LL + (threadIdx.x >> 5); r < mats * rows_p; r += gridDim.x * 8LL) {
    const int64_t m = r / rows_p, rr = r - m * rows_p;
    const __nv_bfloat16* q = in + (m * rows + min(rr, rows - 1)) * cols;
    for (int64_t c = lane * 8; c < cols_p; c += 256) {
      const int n = rr < rows ? static_cast<int>(min(cols - c, static_cast<int64_t>(8))) : 0;
      *reinterpret_cast<uint4*>(out + r * cols_p + c) = load8(q + c, n, false);
    }
  }
}

namespace {

// CTAs that are resident at once: clusters of four do not fill every GPC.
template <int KIND, int PAIRS>
int resident_ctas(int sms, int smem) {
  if (PAIRS == 1) return sms / 2 * 2;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(sms / 4 * 4), c.blockDim = dim3(kThreads), c.dynamicSmemBytes = smem;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = 2 * PAIRS, at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
  c.attrs = &at, c.numAttrs = 1;
  int n = 0;
  const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, ex_gemm_kernel<KIND, PAIRS>, &c);
  if (e != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    return sms / 4 * 4;      // the last clusters then start late
  }
  return n * 2 * PAIRS;
}

template <int KIND, int PAIRS>
cudaError_t gemm_launch(ExGemmParams p, int sms, bool early, cudaStream_t s) {
  p.inject = take_injected_stall(kInjectGemm);
  p.stages = kMostStages;
  if (gemm_smem(KIND, p.stages, p.experts) > kSmemLimit) p.stages = kMostStages - 1;
  const int smem = gemm_smem(KIND, p.stages, p.experts);
  const cudaError_t e = cudaFuncSetAttribute(ex_gemm_kernel<KIND, PAIRS>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_after(ex_gemm_kernel<KIND, PAIRS>, resident_ctas<KIND, PAIRS>(sms, smem), kThreads, smem, early, s, p);
}

template <int KIND>
cudaError_t gemm_pairs(const ExGemmParams& p, int sms, bool early, cudaStream_t s) {
  return p.pairs == 2 ? gemm_launch<KIND, 2>(p, sms, early, s) : gemm_launch<KIND, 1>(p, sms, early, s);
}

unsigned some(int64_t n, int64_t most) { return static_cast<unsigned>(std::min(std::max<int64_t>(n, 1), most)); }

}  // namespace

cudaError_t launch_ex_gemm(int kind, const ExGemmParams& p, int sms, bool early, cudaStream_t s) {
  switch (kind) {
    case kExUp: return gemm_pairs<kExUp>(p, sms, early, s);
    case kExDown: return gemm_pairs<kExDown>(p, sms, early, s);
    case kExDact: return gemm_launch<kExDact, 1>(p, sms, early, s);
    case kExDx: return gemm_pairs<kExDx>(p, sms, early, s);
    case kExDwIn: return gemm_pairs<kExDwIn>(p, sms, early, s);
    default: return gemm_pairs<kExDwOut>(p, sms, early, s);
  }
}

cudaError_t launch_ex_spread(ExSpreadParams p, int blocks, cudaStream_t s) {
  // the products' split of the SM's memory: an SM changes it only when idle, and
  // a product is to start beside this kernel
  const cudaError_t e = cudaFuncSetAttribute(ex_spread_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                             cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  // few tokens: more warps, each with one load a lane
  p.span = p.tokens >= int64_t{4} * blocks ? 2048 : 256;
  const unsigned pieces = static_cast<unsigned>((p.hp + p.span - 1) / p.span);
  const dim3 grid(some((p.tokens + 7) / 8, std::max(1, blocks / static_cast<int>(pieces))), pieces);
  return launch_after(ex_spread_kernel, grid, 256, 3 * (p.experts + 1) * sizeof(int), p.beside != 0, s, p);
}

cudaError_t launch_ex_combine(const ExCombineParams& p, int sms, bool early, cudaStream_t s) {
  const unsigned warps = some((p.hidden + 255) / 256, 8), block = warps * 32;
  const unsigned grid = some(p.tokens, static_cast<int64_t>(sms) * (24 / warps));
  if (p.top_k == 1) return launch_after(ex_combine_kernel<1>, grid, block, 0, early, s, p);
  if (p.top_k == 2) return launch_after(ex_combine_kernel<2>, grid, block, 0, early, s, p);
  if (p.top_k <= 4) return launch_after(ex_combine_kernel<4>, grid, block, 0, early, s, p);
  return launch_after(ex_combine_kernel<8>, grid, block, 0, early, s, p);
}

cudaError_t launch_ex_dweights(const ExWeightParams& p, bool early, cudaStream_t s) {
  return launch_after(ex_dweights_kernel, some((p.rows + 255) / 256, 1 << 16), 256, 0, early, s, p);
}

cudaError_t launch_ex_repack(const __nv_bfloat16* in, int64_t mats, int64_t rows, int64_t cols,
                             __nv_bfloat16* out, int64_t rows_p, int64_t cols_p, cudaStream_t s) {
  ex_repack_kernel<<<some((mats * rows_p + 7) / 8, 1 << 14), 256, 0, s>>>(in, mats, rows, cols, out, rows_p,
                                                                         cols_p);
  return cudaGetLastError();
}

}  // namespace muon
