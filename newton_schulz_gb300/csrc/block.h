// Internal interface of the mixture-of-experts block's operators (RMS norm,
// routing, experts' products) between their host side (block_api.cpp) and
// their kernels.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>
#include <type_traits>
#include <vector>

#include "muon_internal.h"

namespace muon {

// ---- library state owned by api.cpp ---------------------------------------------------
struct ApiDevice {
  int sms;
  unsigned* status;                  // device status word
  unsigned long long timeout_ns;     // bound of a device wait
};
// All are called with api_mutex() held.  api_workspace: at least `bytes`
// bytes of the (device, stream) workspace, whose contents last until the next
// call on that stream.  api_guard_bytes: size of the band behind every buffer in
// guard mode (MUON_WS_GUARD), else 0; bands are filled before the call's launches
// and checked after them.
std::mutex& api_mutex();
int api_device(ApiDevice* out);                                          // muon_status_t
int api_workspace(cudaStream_t stream, size_t bytes, char** out);        // muon_status_t
size_t api_guard_bytes();
int api_guard_fill(char* ws, const std::vector<size_t>& bands, cudaStream_t stream);    // muon_status_t
int api_guard_check(char* ws, const std::vector<size_t>& bands, cudaStream_t stream);   // muon_status_t
void api_set_launches(int n);

// Launch of a kernel that follows another of the same call.  early: it may
// start while that one ends (programmatic dependent launch), and waits for its
// results with ptx::wait_dependency before it touches what the call's kernels
// share.  That saves 2 to 4 us a launch (one token through the experts' products
// 26.8 -> 21.3 us, 7 tokens' gradient in eight launches 89 -> 52), also where the
// kernels are long but their rows few (2 of 8 x [14336, 4096]: 34 rows 456 -> 446,
// 4096 rows 951 -> 944); under many rows the waiting blocks take room from the
// running ones (the products' gradient over 64 experts 1247 -> 1266 us).
template <typename... A>
cudaError_t launch_after(void (*kernel)(A...), dim3 grid, unsigned block, size_t smem, bool early,
                         cudaStream_t s, typename std::common_type<A>::type... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- RMS norm --------------------------------------------------------------------------
constexpr int kNormMaxCols = 32768;
constexpr int kDtF32 = 0, kDtBf16 = 1, kDtE4m3 = 2, kDtNone = -1;

struct NormParams {
  const void* x;
  const void* res;
  const void* gain;
  void* h;
  void* y;
  float* scales;
  int64_t rows, xs, rs, hs, ys;
  int cols;
  int x_dt, r_dt, g_dt, h_dt, y_dt;   // kDt*; kDtNone: absent
  int grouped;                        // e4m3: a scale per 128 columns (0: per row)
  int n_scales;                       // scales per row
  int vec;                            // 16-byte accesses are legal
  float eps, inv_cols;                // inv_cols = 1 / cols
  unsigned* status;
};

struct NormGradParams {
  const void* dy;
  const void* h;
  const void* gain;
  const void* dres;
  void* dh;
  float* part;                        // [slots][cols] partial dgain, or null
  int64_t rows, dys, hs, drs, dhs;
  int cols;
  int dy_dt, h_dt, g_dt, dr_dt, dh_dt;
  int vec;
  float eps, inv_cols;
  unsigned* status;
  unsigned long long timeout_ns;
  int inject;                         // testing hook (set at the launch): row 0 never arrives
};

cudaError_t launch_norm(const NormParams& p, int sms, cudaStream_t s);
// Row slots (rows of NormGradParams::part) that launch_norm_grad uses for p.
int norm_grad_slots(const NormGradParams& p, int sms);
cudaError_t launch_norm_grad(const NormGradParams& p, int sms, cudaStream_t s);
cudaError_t launch_norm_dgain(const float* part, int slots, int cols, float* dgain, cudaStream_t s);

// ---- routing ----------------------------------------------------------------------------
constexpr int kRouteMaxExperts = 1024, kRouteMaxTopK = 32, kRouteMaxGroups = 64;
constexpr int kPlanTokens = 256;      // tokens per tile of the plan's counting sort

struct RouteParams {
  const void* logits;
  int64_t stride, tokens;
  int dtype;
  const float* bias;
  const uint8_t* mask;
  int32_t* idx;
  float* weights;
  int experts, top_k, score, groups, top_groups, group_score, renorm;
  int vec, bias_vec;              // 16-byte aligned rows of logits, bias
  float scale;
  unsigned* status;
};

struct RouteGradParams {
  const void* logits;
  int64_t stride, tokens, dstride;
  int dtype;
  const int32_t* idx;
  const float* dweights;
  void* dlogits;
  int experts, top_k, score, renorm;
  int vec, dvec;                  // 16-byte aligned rows of logits, dlogits
  float scale;
  unsigned* status;
};

struct PlanParams {
  const int32_t* idx;
  int64_t tokens;
  int top_k, experts;
  int tiles;                // ceil(tokens / kPlanTokens)
  int32_t* hist;            // [tiles][experts] (workspace; unused with one tile)
  int32_t* offsets;
  int32_t* src;
  int32_t* pos;
  unsigned* status;
};

cudaError_t launch_route(const RouteParams& p, cudaStream_t s);
cudaError_t launch_route_grad(const RouteGradParams& p, cudaStream_t s);
cudaError_t launch_plan_hist(const PlanParams& p, bool early, cudaStream_t s);   // early: see launch_after
cudaError_t launch_plan(const PlanParams& p, bool early, cudaStream_t s);

// ---- experts' products ---------------------------------------------------------------------
// Products on the tensor cores (experts.cu), by operand and result.
enum ExKind : int {
  kExUp = 0,     // rows x W_in^T  -> act (and gate, up)
  kExDown = 1,   // act  x W_out^T -> y
  kExDact = 2,   // dout x W_out   -> dgu, w a, dweights' parts
  kExDx = 3,     // dgu  x W_in    -> y
  kExDwIn = 4,   // dgu^T  x rows
  kExDwOut = 5   // dout^T x w a
};
constexpr int kExSeg = 64;        // row segments of the gradient's buffers: a K block
constexpr int kExMTile = 256;     // rows of the weight-side dimension per CTA pair
constexpr int kExNTile = 256;     // most token rows (gradients: columns) per CTA pair

struct ExGemmParams {
  CUtensorMap mapA, mapB;         // weight-side and token-side operand
  CUtensorMap mapB32;             // token rows in boxes of 32 (kExDw*: unused)
  const int32_t* offsets;         // [experts + 1]
  int64_t rows;                   // tokens * top_k, the most rows there are
  int64_t prows;                  // the same in the padded numbering
  int experts;
  int beside;                     // 1: runs beside the previous launch, whose results it does not use
  int pad;                        // padded row numbering: segments of 1 or kExSeg rows
  int m_tiles, n_tiles;           // M tiles of a pair; kExDw*: N tiles
  int kb;                         // K blocks of 64 (kExDw*: from the expert's rows)
  int pairs;                      // CTA pairs per cluster, 1 or 2
  int m, n;                       // valid M (padded for kExDwIn) and, kExDw*, N
  int inner, ip;                  // inner, and rounded up to 8
  int ap, gp;                     // pitches of act and dgu
  __nv_bfloat16* act;             // [padded rows][ap]: kExUp act, kExDact w a
  __nv_bfloat16* gu;              // [rows][2 inner]: kExUp output or null, kExDact input
  int gu_vec;                     // 16-byte accesses to gu are legal
  __half* y;                      // [rows][yp] values scaled by a power of two
  int64_t yp;
  uint8_t* yexp;                  // [rows][yep] exponents, one per 32 columns
  int64_t yep;
  const float* wr;                // [padded rows] weight of a row
  __nv_bfloat16* dgu;             // [padded rows][gp], gate part then up part at ip
  float* part;                    // [features / 32][rows] parts of dweights
  void* dw;
  int dw_dt, dw_vec;
  int stages;                     // ring depth (set at the launch)
  int inject;                     // testing hook (set at the launch): CTA 0's MMA issuer
                                  // waits for what nothing provides
  int a_whole;                    // MN-major weights in one copy of two 64-column chunks
  unsigned* status;
  unsigned long long timeout_ns;
};

// Rows of x (or dout) in expert order, zero rows up to each segment's end.
struct ExSpreadParams {
  const __nv_bfloat16* x;
  int64_t xs;
  __nv_bfloat16* out;             // [padded rows][hp]
  int vec;                        // 16-byte accesses are legal
  const float* weights;           // with wr: the row's weight
  float* wr;
  const int32_t* offsets;
  const int32_t* pos;
  int64_t tokens, rows, hidden, hp;
  int64_t prows;                  // rows of out
  unsigned* status;
  int experts, top_k, pad;
  int span;                       // columns a warp takes at a time (set at the launch)
  int beside;                     // 1: runs beside the previous launch, whose results it does not use
};

struct ExCombineParams {          // out[t] = sum_j w[t,j] y[pos[t,j]]
  const __half* y;                // as ExGemmParams wrote it
  int64_t yp;
  const uint8_t* yexp;
  int64_t yep;
  const int32_t* pos;
  const float* weights;           // null: ones
  __nv_bfloat16* out;
  int64_t outs, tokens, hidden, rows;
  int top_k, vec;
};

struct ExWeightParams {           // dweights[t,j] = sum over parts of part[.][pos[t,j]]
  const float* part;
  const int32_t* pos;
  float* dweights;
  int64_t rows;
  int parts;
};

// A few rows: matrix-vector products, two launches, no padding or copies.
constexpr int kExFewRows = 32;    // most of them; few_rows (block_api.cpp) has the rule
struct ExFewParams {
  const __nv_bfloat16* x;
  int64_t xs;
  const __nv_bfloat16* w_in;      // [experts][2 inner][hidden]
  const __nv_bfloat16* w_out;     // [experts][hidden][inner]
  const float* weights;
  const int32_t* offsets;
  const int32_t* src;
  const int32_t* pos;
  __nv_bfloat16* gu;              // [rows][2 inner] or null
  float* act;                     // [rows][ip], 16-byte aligned rows
  __nv_bfloat16* out;
  int64_t outs, tokens, ip;
  int hidden, inner, experts, top_k, rows;
  int vec_in, vec_out;            // 16-byte loads of x and w_in, of w_out
  unsigned* status;
};
cudaError_t launch_ex_few(const ExFewParams& p, cudaStream_t s);    // two launches

// early: see launch_after
cudaError_t launch_ex_gemm(int kind, const ExGemmParams& p, int sms, bool early, cudaStream_t s);
cudaError_t launch_ex_spread(ExSpreadParams p, int blocks, cudaStream_t s);
cudaError_t launch_ex_combine(const ExCombineParams& p, int sms, bool early, cudaStream_t s);
cudaError_t launch_ex_dweights(const ExWeightParams& p, bool early, cudaStream_t s);
// mats matrices [rows][cols] -> [rows_p][cols_p], zeros around
cudaError_t launch_ex_repack(const __nv_bfloat16* in, int64_t mats, int64_t rows, int64_t cols,
                             __nv_bfloat16* out, int64_t rows_p, int64_t cols_p, cudaStream_t s);

}  // namespace muon
