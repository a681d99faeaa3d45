// C ABI of the mixture-of-experts block's operators: argument checks,
// workspace layout and launches (include/muon.h has their definitions).
#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>

#include "../../include/muon.h"
#include "block.h"

using namespace muon;

namespace {

bool is_float_dtype(int dt) { return dt == MUON_F32 || dt == MUON_BF16; }
int64_t esize(int dt) { return dt == MUON_F32 ? 4 : dt == MUON_BF16 ? 2 : 1; }
bool aligned(const void* p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
size_t pad256(size_t n) { return (n + 255) / 256 * 256; }

// A [rows, cols] tensor argument with a row stride, in elements.
struct View {
  const void* p;
  int dt;
  int64_t rows, cols, stride;
  uintptr_t lo() const { return reinterpret_cast<uintptr_t>(p); }
  uintptr_t hi() const {
    return rows <= 0 ? lo() : lo() + static_cast<uintptr_t>(((rows - 1) * stride + cols) * esize(dt));
  }
  bool overlaps(const View& o) const { return p && o.p && lo() < o.hi() && o.lo() < hi(); }
  bool same(const View& o) const { return p == o.p && dt == o.dt && (stride == o.stride || rows <= 1); }
  bool bad_stride() const { return rows > 1 && (stride < cols || stride > (int64_t(1) << 40)); }
  // every row starts on a 16-byte boundary
  bool rows16() const { return !p || (aligned(p, 16) && (rows <= 1 || stride * esize(dt) % 16 == 0)); }
};

View dense(const void* p, int dt, int64_t n) { return View{p, dt, 1, n, n}; }

struct Counter {
  int n = 0;
  muon_status_t run(cudaError_t e) {
    if (e != cudaSuccess) return MUON_ERR_CUDA;
    ++n;
    return MUON_OK;
  }
};

#define MUON_TRY(expr)                              \
  do {                                              \
    const muon_status_t st_ = (expr);               \
    if (st_ != MUON_OK) return st_;                 \
  } while (0)

muon_status_t device(ApiDevice* d) { return static_cast<muon_status_t>(api_device(d)); }
muon_status_t workspace(cudaStream_t s, size_t n, char** out) {
  return static_cast<muon_status_t>(api_workspace(s, n, out));
}

// ---- RMS norm --------------------------------------------------------------------------
muon_status_t norm_impl(const muon_rmsnorm_t* a, cudaStream_t stream) {
  if (!a || a->rows < 0 || a->cols < 0) return MUON_ERR_INVALID_ARGUMENT;
  const bool e4m3 = a->y_dtype == MUON_E4M3;
  if (!is_float_dtype(a->x_dtype) || !(is_float_dtype(a->y_dtype) || e4m3) ||
      (a->residual && !is_float_dtype(a->residual_dtype)) || (a->gain && !is_float_dtype(a->gain_dtype)) ||
      (a->h && !is_float_dtype(a->h_dtype)))
    return MUON_ERR_INVALID_ARGUMENT;
  if (!(a->eps >= 0.f) || !std::isfinite(a->eps)) return MUON_ERR_INVALID_ARGUMENT;
  if (a->group != 0 && !(e4m3 && a->group == 128)) return MUON_ERR_INVALID_ARGUMENT;
  if (a->rows == 0 || a->cols == 0) {
    api_set_launches(0);
    return MUON_OK;
  }
  if (a->cols > kNormMaxCols || a->rows > 0x7fffffff) return MUON_ERR_UNSUPPORTED;
  if (!a->x || !a->y || (e4m3 && !a->scales)) return MUON_ERR_INVALID_ARGUMENT;
  const int64_t n_scales = a->group ? (a->cols + a->group - 1) / a->group : 1;
  const View x{a->x, a->x_dtype, a->rows, a->cols, a->x_stride},
      r{a->residual, a->residual_dtype, a->rows, a->cols, a->residual_stride},
      h{a->h, a->h_dtype, a->rows, a->cols, a->h_stride}, y{a->y, a->y_dtype, a->rows, a->cols, a->y_stride},
      g = dense(a->gain, a->gain_dtype, a->cols),
      sc = dense(e4m3 ? a->scales : nullptr, MUON_F32, a->rows * n_scales);
  for (const View* v : {&x, &r, &h, &y, &g, &sc}) {
    if (!v->p) continue;
    if (v->bad_stride() || !aligned(v->p, esize(v->dt))) return MUON_ERR_INVALID_ARGUMENT;
  }
  for (const View* o : {&h, &y, &sc})
    for (const View* i : {&x, &r, &g})
      if (o->overlaps(*i) && !(o == &h && i != &g && h.same(*i))) return MUON_ERR_ALIAS;
  if (h.overlaps(y) || h.overlaps(sc) || y.overlaps(sc)) return MUON_ERR_ALIAS;
  NormParams p;
  std::memset(&p, 0, sizeof(p));
  p.x = a->x, p.res = a->residual, p.gain = a->gain, p.h = a->h, p.y = a->y, p.scales = a->scales;
  p.rows = a->rows, p.cols = static_cast<int>(a->cols);
  p.xs = a->x_stride, p.rs = a->residual_stride, p.hs = a->h_stride, p.ys = a->y_stride;
  p.x_dt = a->x_dtype;
  p.r_dt = a->residual ? a->residual_dtype : kDtNone;
  p.g_dt = a->gain ? a->gain_dtype : kDtNone;
  p.h_dt = a->h ? a->h_dtype : kDtNone;
  p.y_dt = a->y_dtype;
  p.group_chunks = a->group / 8;
  p.n_scales = static_cast<int>(n_scales);
  p.eps = a->eps;
  p.vec = x.rows16() && r.rows16() && h.rows16() && y.rows16() && g.rows16();
  std::lock_guard<std::mutex> lock(api_mutex());
  ApiDevice d;
  MUON_TRY(device(&d));
  Counter c;
  MUON_TRY(c.run(launch_norm(p, d.sms, stream)));
  api_set_launches(c.n);
  return MUON_OK;
}

muon_status_t norm_grad_impl(const muon_rmsnorm_grad_t* a, cudaStream_t stream) {
  if (!a || a->rows < 0 || a->cols < 0) return MUON_ERR_INVALID_ARGUMENT;
  if (!is_float_dtype(a->dy_dtype) || !is_float_dtype(a->h_dtype) || !is_float_dtype(a->dh_dtype) ||
      (a->dres && !is_float_dtype(a->dres_dtype)) || (a->gain && !is_float_dtype(a->gain_dtype)))
    return MUON_ERR_INVALID_ARGUMENT;
  if (!(a->eps >= 0.f) || !std::isfinite(a->eps)) return MUON_ERR_INVALID_ARGUMENT;
  if (a->cols > kNormMaxCols || a->rows > 0x7fffffff) return MUON_ERR_UNSUPPORTED;
  if (a->dgain && !aligned(a->dgain, 4)) return MUON_ERR_INVALID_ARGUMENT;
  if (a->rows == 0 || a->cols == 0) {
    api_set_launches(0);
    if (a->dgain && a->cols > 0 &&
        cudaMemsetAsync(a->dgain, 0, static_cast<size_t>(a->cols) * 4, stream) != cudaSuccess)
      return MUON_ERR_CUDA;
    return MUON_OK;
  }
  if (!a->dy || !a->h || !a->dh) return MUON_ERR_INVALID_ARGUMENT;
  const View dy{a->dy, a->dy_dtype, a->rows, a->cols, a->dy_stride},
      h{a->h, a->h_dtype, a->rows, a->cols, a->h_stride},
      dr{a->dres, a->dres_dtype, a->rows, a->cols, a->dres_stride},
      dh{a->dh, a->dh_dtype, a->rows, a->cols, a->dh_stride}, g = dense(a->gain, a->gain_dtype, a->cols),
      dg = dense(a->dgain, MUON_F32, a->cols);
  for (const View* v : {&dy, &h, &dr, &dh, &g}) {
    if (!v->p) continue;
    if (v->bad_stride() || !aligned(v->p, esize(v->dt))) return MUON_ERR_INVALID_ARGUMENT;
  }
  for (const View* i : {&dy, &h, &dr, &g}) {
    if (dh.overlaps(*i) && !((i == &dy || i == &dr) && dh.same(*i))) return MUON_ERR_ALIAS;
    if (dg.overlaps(*i)) return MUON_ERR_ALIAS;
  }
  if (dh.overlaps(dg)) return MUON_ERR_ALIAS;
  NormGradParams p;
  std::memset(&p, 0, sizeof(p));
  p.dy = a->dy, p.h = a->h, p.gain = a->gain, p.dres = a->dres, p.dh = a->dh;
  p.rows = a->rows, p.cols = static_cast<int>(a->cols);
  p.dys = a->dy_stride, p.hs = a->h_stride, p.drs = a->dres_stride, p.dhs = a->dh_stride;
  p.dy_dt = a->dy_dtype, p.h_dt = a->h_dtype, p.dh_dt = a->dh_dtype;
  p.g_dt = a->gain ? a->gain_dtype : kDtNone;
  p.dr_dt = a->dres ? a->dres_dtype : kDtNone;
  p.eps = a->eps;
  p.vec = dy.rows16() && h.rows16() && dr.rows16() && dh.rows16() && g.rows16();
  std::lock_guard<std::mutex> lock(api_mutex());
  ApiDevice d;
  MUON_TRY(device(&d));
  Counter c;
  const int slots = norm_grad_slots(p, d.sms);
  if (a->dgain) {
    char* ws = nullptr;
    MUON_TRY(workspace(stream, static_cast<size_t>(slots) * p.cols * 4, &ws));
    p.part = reinterpret_cast<float*>(ws);
  }
  MUON_TRY(c.run(launch_norm_grad(p, d.sms, stream)));
  if (a->dgain) MUON_TRY(c.run(launch_norm_dgain(p.part, slots, p.cols, a->dgain, stream)));
  api_set_launches(c.n);
  return MUON_OK;
}

// ---- routing ------------------------------------------------------------------------------
bool bad_route_config(const muon_route_config_t* c) {
  return !c || c->experts < 1 || c->top_k < 1 || c->top_k > c->experts ||
         (c->score != MUON_ROUTE_SOFTMAX && c->score != MUON_ROUTE_SIGMOID) || c->groups < 1 ||
         c->groups > c->experts || c->experts % c->groups != 0 || c->top_groups < 1 ||
         c->top_groups > c->groups ||
         (c->group_score != MUON_GROUP_MAX && c->group_score != MUON_GROUP_SUM2) ||
         !std::isfinite(c->scale);
}

bool unsupported_route(int64_t tokens, int top_k, int experts, int groups) {
  return experts > kRouteMaxExperts || top_k > kRouteMaxTopK || groups > kRouteMaxGroups ||
         tokens > 0x7fffffff || tokens * top_k > 0x7fffffff;
}

// The plan's launches; hist: workspace, unused with one tile.
muon_status_t plan_launches(const PlanParams& p, Counter* c, cudaStream_t stream) {
  if (p.tiles > 1) MUON_TRY(c->run(launch_plan_hist(p, stream)));
  return c->run(launch_plan(p, stream));
}

PlanParams plan_params(const int32_t* idx, int64_t tokens, int top_k, int experts, int32_t* offsets,
                       int32_t* src, int32_t* pos) {
  PlanParams p;
  std::memset(&p, 0, sizeof(p));
  p.idx = idx, p.tokens = tokens, p.top_k = top_k, p.experts = experts;
  p.tiles = static_cast<int>((tokens + kPlanTokens - 1) / kPlanTokens);
  p.offsets = offsets, p.src = src, p.pos = pos;
  return p;
}

muon_status_t zero_offsets(int32_t* offsets, int experts, cudaStream_t stream) {
  api_set_launches(0);
  if (!offsets) return MUON_OK;
  return cudaMemsetAsync(offsets, 0, static_cast<size_t>(experts + 1) * 4, stream) == cudaSuccess
             ? MUON_OK
             : MUON_ERR_CUDA;
}

muon_status_t route_impl(const muon_route_config_t* cfg, const void* logits, int dtype, int64_t stride,
                         int64_t tokens, const float* bias, const uint8_t* mask, int32_t* idx,
                         float* weights, int32_t* offsets, int32_t* src, int32_t* pos,
                         cudaStream_t stream) {
  if (bad_route_config(cfg) || tokens < 0 || !is_float_dtype(dtype)) return MUON_ERR_INVALID_ARGUMENT;
  if (unsupported_route(tokens, cfg->top_k, cfg->experts, cfg->groups)) return MUON_ERR_UNSUPPORTED;
  if (!aligned(offsets, 4)) return MUON_ERR_INVALID_ARGUMENT;
  if (tokens == 0) return zero_offsets(offsets, cfg->experts, stream);
  const int64_t picks = tokens * cfg->top_k;
  if (!logits || !idx || !weights || (offsets && (!src || !pos))) return MUON_ERR_INVALID_ARGUMENT;
  const View l{logits, dtype, tokens, cfg->experts, stride}, b = dense(bias, MUON_F32, cfg->experts),
      m = dense(mask, MUON_E4M3, tokens), oi = dense(idx, MUON_F32, picks), ow = dense(weights, MUON_F32, picks),
      oo = dense(offsets, MUON_F32, cfg->experts + 1), os = dense(offsets ? src : nullptr, MUON_F32, picks),
      op = dense(offsets ? pos : nullptr, MUON_F32, picks);
  for (const View* v : {&l, &b, &m, &oi, &ow, &oo, &os, &op})
    if (v->p && (v->bad_stride() || !aligned(v->p, esize(v->dt)))) return MUON_ERR_INVALID_ARGUMENT;
  const View* outs[] = {&oi, &ow, &oo, &os, &op};
  for (int i = 0; i < 5; ++i) {
    for (const View* in : {&l, &b, &m})
      if (outs[i]->overlaps(*in)) return MUON_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (outs[i]->overlaps(*outs[j])) return MUON_ERR_ALIAS;
  }
  std::lock_guard<std::mutex> lock(api_mutex());
  ApiDevice d;
  MUON_TRY(device(&d));
  RouteParams p;
  std::memset(&p, 0, sizeof(p));
  p.logits = logits, p.stride = stride, p.tokens = tokens, p.dtype = dtype;
  p.bias = bias, p.mask = mask, p.idx = idx, p.weights = weights;
  p.experts = cfg->experts, p.top_k = cfg->top_k, p.score = cfg->score, p.groups = cfg->groups;
  p.top_groups = cfg->top_groups, p.group_score = cfg->group_score, p.renorm = cfg->renormalize != 0;
  p.scale = cfg->scale;
  p.status = d.status;
  PlanParams pp = plan_params(idx, tokens, cfg->top_k, cfg->experts, offsets, src, pos);
  if (offsets && pp.tiles > 1) {
    char* ws = nullptr;
    MUON_TRY(workspace(stream, static_cast<size_t>(pp.tiles) * cfg->experts * 4, &ws));
    pp.hist = reinterpret_cast<int32_t*>(ws);
  }
  Counter c;
  MUON_TRY(c.run(launch_route(p, stream)));
  if (offsets) MUON_TRY(plan_launches(pp, &c, stream));
  api_set_launches(c.n);
  return MUON_OK;
}

muon_status_t plan_impl(const int32_t* idx, int64_t tokens, int top_k, int experts, int32_t* offsets,
                        int32_t* src, int32_t* pos, cudaStream_t stream) {
  if (tokens < 0 || top_k < 1 || experts < 1 || !offsets || !aligned(offsets, 4))
    return MUON_ERR_INVALID_ARGUMENT;
  if (unsupported_route(tokens, top_k, experts, 1)) return MUON_ERR_UNSUPPORTED;
  if (tokens == 0) return zero_offsets(offsets, experts, stream);
  if (!idx || !src || !pos) return MUON_ERR_INVALID_ARGUMENT;
  const int64_t picks = tokens * top_k;
  const View i = dense(idx, MUON_F32, picks), o = dense(offsets, MUON_F32, experts + 1),
             s = dense(src, MUON_F32, picks), q = dense(pos, MUON_F32, picks);
  for (const View* v : {&i, &o, &s, &q})
    if (!aligned(v->p, 4)) return MUON_ERR_INVALID_ARGUMENT;
  if (i.overlaps(o) || i.overlaps(s) || i.overlaps(q) || o.overlaps(s) || o.overlaps(q) || s.overlaps(q))
    return MUON_ERR_ALIAS;
  std::lock_guard<std::mutex> lock(api_mutex());
  PlanParams p = plan_params(idx, tokens, top_k, experts, offsets, src, pos);
  if (p.tiles > 1) {
    char* ws = nullptr;
    MUON_TRY(workspace(stream, static_cast<size_t>(p.tiles) * experts * 4, &ws));
    p.hist = reinterpret_cast<int32_t*>(ws);
  }
  Counter c;
  MUON_TRY(plan_launches(p, &c, stream));
  api_set_launches(c.n);
  return MUON_OK;
}

muon_status_t route_grad_impl(const muon_route_config_t* cfg, const void* logits, int dtype,
                              int64_t stride, int64_t tokens, const int32_t* idx, const float* dweights,
                              void* dlogits, int64_t dstride, cudaStream_t stream) {
  if (bad_route_config(cfg) || tokens < 0 || !is_float_dtype(dtype)) return MUON_ERR_INVALID_ARGUMENT;
  if (unsupported_route(tokens, cfg->top_k, cfg->experts, cfg->groups)) return MUON_ERR_UNSUPPORTED;
  if (tokens == 0) {
    api_set_launches(0);
    return MUON_OK;
  }
  if (!logits || !idx || !dweights || !dlogits) return MUON_ERR_INVALID_ARGUMENT;
  const int64_t picks = tokens * cfg->top_k;
  const View l{logits, dtype, tokens, cfg->experts, stride}, o{dlogits, dtype, tokens, cfg->experts, dstride},
      i = dense(idx, MUON_F32, picks), w = dense(dweights, MUON_F32, picks);
  for (const View* v : {&l, &o, &i, &w})
    if (v->bad_stride() || !aligned(v->p, esize(v->dt))) return MUON_ERR_INVALID_ARGUMENT;
  if (o.overlaps(l) || o.overlaps(i) || o.overlaps(w)) return MUON_ERR_ALIAS;
  RouteGradParams p;
  std::memset(&p, 0, sizeof(p));
  p.logits = logits, p.stride = stride, p.tokens = tokens, p.dstride = dstride, p.dtype = dtype;
  p.idx = idx, p.dweights = dweights, p.dlogits = dlogits;
  p.experts = cfg->experts, p.top_k = cfg->top_k, p.score = cfg->score;
  p.renorm = cfg->renormalize != 0;
  p.scale = cfg->scale;
  std::lock_guard<std::mutex> lock(api_mutex());
  Counter c;
  MUON_TRY(c.run(launch_route_grad(p, stream)));
  api_set_launches(c.n);
  return MUON_OK;
}

// ---- experts' products ------------------------------------------------------------------
struct ExpertsViews {
  View x, w_in, w_out, w, off, src, pos;
};

// Checks the common arguments; *empty: nothing to compute.
muon_status_t check_experts(const muon_experts_t* a, ExpertsViews* v, bool* empty) {
  if (!a || a->tokens < 0 || a->hidden < 1 || a->inner < 1 || a->experts < 1 || a->top_k < 1)
    return MUON_ERR_INVALID_ARGUMENT;
  if (unsupported_route(a->tokens, a->top_k, a->experts, 1) || a->hidden > 65536 || a->inner > 65536)
    return MUON_ERR_UNSUPPORTED;
  *empty = a->tokens == 0;
  const int64_t per = a->inner * a->hidden, picks = a->tokens * a->top_k;
  v->x = View{a->x, MUON_BF16, a->tokens, a->hidden, a->x_stride};
  v->w_in = dense(a->w_in, MUON_BF16, 2 * per * a->experts);
  v->w_out = dense(a->w_out, MUON_BF16, per * a->experts);
  v->w = dense(a->weights, MUON_F32, picks);
  v->off = dense(a->offsets, MUON_F32, a->experts + 1);
  v->src = dense(a->src, MUON_F32, picks);
  v->pos = dense(a->pos, MUON_F32, picks);
  if (*empty) return MUON_OK;
  for (const View* i : {&v->x, &v->w_in, &v->w_out, &v->w, &v->off, &v->src, &v->pos})
    if (!i->p || i->bad_stride() || !aligned(i->p, esize(i->dt))) return MUON_ERR_INVALID_ARGUMENT;
  return MUON_OK;
}

// Whether an output overlaps an input or another output.
bool experts_alias(const ExpertsViews& v, std::initializer_list<View> more_inputs,
                   std::initializer_list<View> outputs) {
  for (auto o = outputs.begin(); o != outputs.end(); ++o) {
    for (const View* i : {&v.x, &v.w_in, &v.w_out, &v.w, &v.off, &v.src, &v.pos})
      if (o->overlaps(*i)) return true;
    for (const View& i : more_inputs)
      if (o->overlaps(i)) return true;
    for (auto q = outputs.begin(); q != o; ++q)
      if (o->overlaps(*q)) return true;
  }
  return false;
}

ExpertsParams experts_params(const muon_experts_t* a) {
  ExpertsParams p;
  std::memset(&p, 0, sizeof(p));
  p.tokens = a->tokens, p.hidden = a->hidden, p.inner = a->inner, p.rows = a->tokens * a->top_k;
  p.experts = a->experts, p.top_k = a->top_k;
  p.x = static_cast<const __nv_bfloat16*>(a->x), p.xs = a->x_stride;
  p.w_in = static_cast<const __nv_bfloat16*>(a->w_in);
  p.w_out = static_cast<const __nv_bfloat16*>(a->w_out);
  p.weights = a->weights, p.offsets = a->offsets, p.src = a->src, p.pos = a->pos;
  return p;
}

muon_status_t experts_impl(const muon_experts_t* a, void* out, int64_t outs, void* gu, cudaStream_t stream) {
  ExpertsViews v;
  bool empty = false;
  MUON_TRY(check_experts(a, &v, &empty));
  if (empty) {
    api_set_launches(0);
    return MUON_OK;
  }
  const int64_t rows = a->tokens * a->top_k;
  const View o{out, MUON_BF16, a->tokens, a->hidden, outs}, og = dense(gu, MUON_BF16, rows * 2 * a->inner);
  if (!out || o.bad_stride() || !aligned(out, 2) || !aligned(gu, 2)) return MUON_ERR_INVALID_ARGUMENT;
  if (experts_alias(v, {}, {o, og})) return MUON_ERR_ALIAS;
  ExpertsParams p = experts_params(a);
  std::lock_guard<std::mutex> lock(api_mutex());
  const size_t n_gu = gu ? 0 : pad256(static_cast<size_t>(rows * 2 * a->inner) * 2),
               n_act = pad256(static_cast<size_t>(rows * a->inner) * 2),
               n_y = pad256(static_cast<size_t>(rows * a->hidden) * 2);
  char* ws = nullptr;
  MUON_TRY(workspace(stream, n_gu + n_act + n_y, &ws));
  p.gu = static_cast<__nv_bfloat16*>(gu ? gu : ws);
  p.act = reinterpret_cast<__nv_bfloat16*>(ws + n_gu);
  p.y = reinterpret_cast<__nv_bfloat16*>(ws + n_gu + n_act);
  Counter c;
  MUON_TRY(c.run(launch_experts_gu(p, stream)));
  MUON_TRY(c.run(launch_experts_act(p, stream)));
  MUON_TRY(c.run(launch_experts_down(p, stream)));
  MUON_TRY(c.run(launch_experts_combine(p, p.y, true, static_cast<__nv_bfloat16*>(out), outs, stream)));
  api_set_launches(c.n);
  return MUON_OK;
}

muon_status_t experts_grad_impl(const muon_experts_t* a, const void* dout, int64_t dos, const void* gu,
                                void* dx, int64_t dxs, void* dw_in, void* dw_out, int dw_dt,
                                float* dweights, cudaStream_t stream) {
  ExpertsViews v;
  bool empty = false;
  MUON_TRY(check_experts(a, &v, &empty));
  if (!is_float_dtype(dw_dt)) return MUON_ERR_INVALID_ARGUMENT;
  const int64_t rows = a->tokens * a->top_k, per = a->inner * a->hidden;
  const View vd{dout, MUON_BF16, a->tokens, a->hidden, dos}, vg = dense(gu, MUON_BF16, rows * 2 * a->inner),
             ox{dx, MUON_BF16, a->tokens, a->hidden, dxs}, oi = dense(dw_in, dw_dt, 2 * per * a->experts),
             oo = dense(dw_out, dw_dt, per * a->experts), ow = dense(dweights, MUON_F32, rows);
  for (const View* o : {&vd, &vg, &ox, &oi, &oo, &ow})
    if (o->p && (o->bad_stride() || !aligned(o->p, esize(o->dt)))) return MUON_ERR_INVALID_ARGUMENT;
  if (!empty && (!dout || !gu)) return MUON_ERR_INVALID_ARGUMENT;
  if (experts_alias(v, {vd, vg}, {ox, oi, oo, ow})) return MUON_ERR_ALIAS;
  Counter c;
  if (empty) {   // no rows: zero weight gradients
    for (const View* o : {&oi, &oo})
      if (o->p && cudaMemsetAsync(const_cast<void*>(o->p), 0, static_cast<size_t>(o->cols * esize(o->dt)),
                                  stream) != cudaSuccess)
        return MUON_ERR_CUDA;
    api_set_launches(0);
    return MUON_OK;
  }
  ExpertsParams p = experts_params(a);
  p.dout = static_cast<const __nv_bfloat16*>(dout), p.dos = dos;
  p.gu_in = static_cast<const __nv_bfloat16*>(gu);
  p.dx = static_cast<__nv_bfloat16*>(dx), p.dxs = dxs;
  p.dw_in = dw_in, p.dw_out = dw_out, p.dw_dt = dw_dt, p.dweights = dweights;
  std::lock_guard<std::mutex> lock(api_mutex());
  const size_t n_da = pad256(static_cast<size_t>(rows * a->inner) * 4),
               n_dgu = pad256(static_cast<size_t>(rows * 2 * a->inner) * 2),
               n_wa = pad256(static_cast<size_t>(rows * a->inner) * 2),
               n_dx = dx ? pad256(static_cast<size_t>(rows * a->hidden) * 2) : 0;
  char* ws = nullptr;
  MUON_TRY(workspace(stream, n_da + n_dgu + n_wa + n_dx, &ws));
  p.da = reinterpret_cast<float*>(ws);
  p.dgu = reinterpret_cast<__nv_bfloat16*>(ws + n_da);
  p.wact = reinterpret_cast<__nv_bfloat16*>(ws + n_da + n_dgu);
  p.dxr = reinterpret_cast<__nv_bfloat16*>(ws + n_da + n_dgu + n_wa);
  if (dweights && cudaMemsetAsync(dweights, 0, static_cast<size_t>(rows) * 4, stream) != cudaSuccess)
    return MUON_ERR_CUDA;
  MUON_TRY(c.run(launch_experts_da(p, stream)));
  MUON_TRY(c.run(launch_experts_dact(p, stream)));
  if (dx) {
    MUON_TRY(c.run(launch_experts_dx(p, stream)));
    MUON_TRY(c.run(launch_experts_combine(p, p.dxr, false, p.dx, dxs, stream)));
  }
  if (dw_in) MUON_TRY(c.run(launch_experts_dw(p, false, stream)));
  if (dw_out) MUON_TRY(c.run(launch_experts_dw(p, true, stream)));
  api_set_launches(c.n);
  return MUON_OK;
}

template <typename F>
muon_status_t guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return MUON_ERR_OUT_OF_MEMORY;
  }
}

}  // namespace

extern "C" {

muon_status_t muon_rmsnorm_forward(const muon_rmsnorm_t* args, cudaStream_t stream) {
  return guarded([&] { return norm_impl(args, stream); });
}

muon_status_t muon_rmsnorm_backward(const muon_rmsnorm_grad_t* args, cudaStream_t stream) {
  return guarded([&] { return norm_grad_impl(args, stream); });
}

muon_status_t muon_route_forward(const muon_route_config_t* cfg, const void* logits, int32_t dtype,
                                 int64_t stride, int64_t tokens, const float* bias, const uint8_t* mask,
                                 int32_t* idx, float* weights, int32_t* offsets, int32_t* src,
                                 int32_t* pos, cudaStream_t stream) {
  return guarded([&] {
    return route_impl(cfg, logits, dtype, stride, tokens, bias, mask, idx, weights, offsets, src, pos, stream);
  });
}

muon_status_t muon_route_plan(const int32_t* idx, int64_t tokens, int32_t top_k, int32_t experts,
                              int32_t* offsets, int32_t* src, int32_t* pos, cudaStream_t stream) {
  return guarded([&] { return plan_impl(idx, tokens, top_k, experts, offsets, src, pos, stream); });
}

muon_status_t muon_route_backward(const muon_route_config_t* cfg, const void* logits, int32_t dtype,
                                  int64_t stride, int64_t tokens, const int32_t* idx,
                                  const float* dweights, void* dlogits, int64_t dlogits_stride,
                                  cudaStream_t stream) {
  return guarded([&] {
    return route_grad_impl(cfg, logits, dtype, stride, tokens, idx, dweights, dlogits, dlogits_stride, stream);
  });
}

muon_status_t muon_experts_forward(const muon_experts_t* args, void* out, int64_t out_stride, void* gu,
                                   cudaStream_t stream) {
  return guarded([&] { return experts_impl(args, out, out_stride, gu, stream); });
}

muon_status_t muon_experts_backward(const muon_experts_t* args, const void* dout, int64_t dout_stride,
                                    const void* gu, void* dx, int64_t dx_stride, void* dw_in,
                                    void* dw_out, int32_t dw_dtype, float* dweights, cudaStream_t stream) {
  return guarded([&] {
    return experts_grad_impl(args, dout, dout_stride, gu, dx, dx_stride, dw_in, dw_out, dw_dtype, dweights,
                             stream);
  });
}

}  // extern "C"
