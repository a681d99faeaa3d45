// Internal interface of the mixture-of-experts block's operators (RMS norm,
// routing, experts' products) between their host side (block_api.cpp) and
// their kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "muon_internal.h"

namespace muon {

// ---- library state owned by api.cpp ---------------------------------------------------
struct ApiDevice {
  int sms;
  unsigned* status;                  // device status word
  unsigned long long timeout_ns;     // bound of a device wait
};
// Both are called with api_mutex() held.  api_workspace: at least `bytes`
// bytes of the (device, stream) workspace, whose contents last until the next
// call on that stream.
std::mutex& api_mutex();
int api_device(ApiDevice* out);                                          // muon_status_t
int api_workspace(cudaStream_t stream, size_t bytes, char** out);        // muon_status_t
void api_set_launches(int n);

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
  int group_chunks;                   // e4m3: 8-column chunks per scale, 0 = the whole row
  int n_scales;                       // scales per row
  int vec;                            // 16-byte accesses are legal
  float eps;
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
  float eps;
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
  float scale;
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
};

cudaError_t launch_route(const RouteParams& p, cudaStream_t s);
cudaError_t launch_route_grad(const RouteGradParams& p, cudaStream_t s);
cudaError_t launch_plan_hist(const PlanParams& p, cudaStream_t s);
cudaError_t launch_plan(const PlanParams& p, cudaStream_t s);

// ---- experts' products ---------------------------------------------------------------------
struct ExpertsParams {
  int64_t tokens, hidden, inner, rows;   // rows = tokens * top_k
  int experts, top_k;
  const __nv_bfloat16* x;
  int64_t xs;
  const __nv_bfloat16* w_in;
  const __nv_bfloat16* w_out;
  const float* weights;
  const int32_t* offsets;
  const int32_t* src;
  const int32_t* pos;
  // forward
  __nv_bfloat16* gu;        // [rows][2 inner]
  __nv_bfloat16* act;       // [rows][inner]
  __nv_bfloat16* y;         // [rows][hidden]
  __nv_bfloat16* out;
  int64_t outs;
  // backward
  const __nv_bfloat16* dout;
  int64_t dos;
  const __nv_bfloat16* gu_in;
  float* da;                // [rows][inner]
  __nv_bfloat16* dgu;       // [rows][2 inner]
  __nv_bfloat16* wact;      // [rows][inner]
  __nv_bfloat16* dxr;       // [rows][hidden]
  __nv_bfloat16* dx;
  int64_t dxs;
  void* dw_in;
  void* dw_out;
  int dw_dt;
  float* dweights;
};

cudaError_t launch_experts_gu(const ExpertsParams& p, cudaStream_t s);
cudaError_t launch_experts_act(const ExpertsParams& p, cudaStream_t s);
cudaError_t launch_experts_down(const ExpertsParams& p, cudaStream_t s);
cudaError_t launch_experts_da(const ExpertsParams& p, cudaStream_t s);
cudaError_t launch_experts_dact(const ExpertsParams& p, cudaStream_t s);
cudaError_t launch_experts_dx(const ExpertsParams& p, cudaStream_t s);
cudaError_t launch_experts_dw(const ExpertsParams& p, bool w_out, cudaStream_t s);
// out[t] = sum_j (weighted ? weights[t,j] : 1) rows[pos[t,j]]
cudaError_t launch_experts_combine(const ExpertsParams& p, const __nv_bfloat16* rows, bool weighted,
                                   __nv_bfloat16* out, int64_t outs, cudaStream_t s);

}  // namespace muon
