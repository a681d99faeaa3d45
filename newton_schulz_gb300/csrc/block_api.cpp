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
  // Whether an element is in both: their spans meet, and they are not different
  // columns of rows one pitch apart (or one row between such rows' columns).
  bool overlaps(const View& o) const {
    if (!p || !o.p || lo() >= o.hi() || o.lo() >= hi()) return false;
    const int64_t pa = stride * esize(dt), pb = o.stride * esize(o.dt);
    if ((rows <= 1 && o.rows <= 1) || (rows > 1 && o.rows > 1 && pa != pb)) return true;
    const int64_t pitch = rows > 1 ? pa : pb, wa = cols * esize(dt), wb = o.cols * esize(o.dt);
    const int64_t d = static_cast<int64_t>(o.lo() - lo()) % pitch, at = d < 0 ? d + pitch : d;
    return at < wa || at + wb > pitch;
  }
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

// Workspace, cut into 256-byte aligned pieces, each followed by a guard band in
// guard mode: sizes first, then pointers, then the launches between open and close.
struct Carve {
  size_t bytes = 0;
  const size_t guard = api_guard_bytes();
  std::vector<size_t> bands;
  char* ws = nullptr;
  size_t take(int64_t n) {
    const size_t at = bytes;
    bytes += pad256(static_cast<size_t>(n));
    if (guard) {
      bands.push_back(bytes);
      bytes += guard;
    }
    return at;
  }
  muon_status_t open(cudaStream_t s) {
    const muon_status_t st = static_cast<muon_status_t>(api_workspace(s, bytes, &ws));
    return st != MUON_OK || !guard ? st : static_cast<muon_status_t>(api_guard_fill(ws, bands, s));
  }
  muon_status_t close(cudaStream_t s) {
    return guard ? static_cast<muon_status_t>(api_guard_check(ws, bands, s)) : MUON_OK;
  }
};

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
  p.grouped = a->group != 0;
  p.n_scales = static_cast<int>(n_scales);
  p.eps = a->eps, p.inv_cols = 1.f / static_cast<float>(a->cols);
  p.vec = x.rows16() && r.rows16() && h.rows16() && y.rows16() && g.rows16();
  std::lock_guard<std::mutex> lock(api_mutex());
  ApiDevice d;
  MUON_TRY(device(&d));
  p.status = d.status;
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
  p.eps = a->eps, p.inv_cols = 1.f / static_cast<float>(a->cols);
  p.vec = dy.rows16() && h.rows16() && dr.rows16() && dh.rows16() && g.rows16();
  std::lock_guard<std::mutex> lock(api_mutex());
  ApiDevice d;
  MUON_TRY(device(&d));
  Counter c;
  p.status = d.status, p.timeout_ns = d.timeout_ns;
  const int slots = norm_grad_slots(p, d.sms);
  Carve cv;
  if (a->dgain) {
    cv.take(static_cast<int64_t>(slots) * p.cols * 4);
    MUON_TRY(cv.open(stream));
    p.part = reinterpret_cast<float*>(cv.ws);
  }
  MUON_TRY(c.run(launch_norm_grad(p, d.sms, stream)));
  if (a->dgain) {
    MUON_TRY(c.run(launch_norm_dgain(p.part, slots, p.cols, a->dgain, stream)));
    MUON_TRY(cv.close(stream));
  }
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
  if (p.tiles > 1) MUON_TRY(c->run(launch_plan_hist(p, c->n > 0, stream)));
  return c->run(launch_plan(p, c->n > 0, stream));
}

muon_status_t plan_counts(PlanParams* p, Carve* cv, cudaStream_t stream) {
  cv->take(static_cast<int64_t>(p->tiles) * p->experts * 4);
  MUON_TRY(cv->open(stream));
  p->hist = reinterpret_cast<int32_t*>(cv->ws);
  return MUON_OK;
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
  p.vec = l.rows16(), p.bias_vec = aligned(bias, 16);
  p.scale = cfg->scale;
  p.status = d.status;
  PlanParams pp = plan_params(idx, tokens, cfg->top_k, cfg->experts, offsets, src, pos);
  pp.status = d.status;
  Carve cv;
  const bool counts = offsets && pp.tiles > 1;
  if (counts) MUON_TRY(plan_counts(&pp, &cv, stream));
  Counter c;
  MUON_TRY(c.run(launch_route(p, stream)));
  if (offsets) MUON_TRY(plan_launches(pp, &c, stream));
  if (counts) MUON_TRY(cv.close(stream));
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
  ApiDevice d;
  MUON_TRY(device(&d));
  PlanParams p = plan_params(idx, tokens, top_k, experts, offsets, src, pos);
  p.status = d.status;
  Carve cv;
  if (p.tiles > 1) MUON_TRY(plan_counts(&p, &cv, stream));
  Counter c;
  MUON_TRY(plan_launches(p, &c, stream));
  if (p.tiles > 1) MUON_TRY(cv.close(stream));
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
  p.vec = l.rows16(), p.dvec = o.rows16();
  p.scale = cfg->scale;
  std::lock_guard<std::mutex> lock(api_mutex());
  ApiDevice d;
  MUON_TRY(device(&d));
  p.status = d.status;
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

int64_t rup(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// The weights as the tensor maps want them: rows of a multiple of 8 elements
// on 16-byte boundaries, inner a multiple of 8 (gate and up rows interleave
// by 8).  Others are copied into the workspace with zeros around.
struct WeightPlan {
  int64_t hp, ip;            // hidden and inner rounded up to 8
  bool pack_in, pack_out;
  size_t at_in, at_out;
  WeightPlan(const muon_experts_t* a, Carve* c)
      : hp(rup(a->hidden, 8)),
        ip(rup(a->inner, 8)),
        pack_in(hp != a->hidden || ip != a->inner || !aligned(a->w_in, 16)),
        pack_out(ip != a->inner || !aligned(a->w_out, 16)) {
    at_in = pack_in ? c->take(2LL * a->experts * ip * hp * 2) : 0;
    at_out = pack_out ? c->take(static_cast<int64_t>(a->experts) * a->hidden * ip * 2) : 0;
  }
};

muon_status_t pack_weights(const muon_experts_t* a, const WeightPlan& w, char* ws, const __nv_bfloat16** w_in,
                           const __nv_bfloat16** w_out, Counter* c, cudaStream_t s) {
  *w_in = static_cast<const __nv_bfloat16*>(a->w_in);
  *w_out = static_cast<const __nv_bfloat16*>(a->w_out);
  if (w.pack_in) {
    __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(ws + w.at_in);
    MUON_TRY(c->run(launch_ex_repack(*w_in, 2LL * a->experts, a->inner, a->hidden, o, w.ip, w.hp, s)));
    *w_in = o;
  }
  if (w.pack_out) {
    __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(ws + w.at_out);
    MUON_TRY(c->run(launch_ex_repack(*w_out, a->experts, a->hidden, a->inner, o, a->hidden, w.ip, s)));
    *w_out = o;
  }
  return MUON_OK;
}

// ---- tensor maps -------------------------------------------------------------------------
// bf16, 128-byte swizzle, rank 2 to 5; strides (bytes) of dims 1 and up.
bool encode_bf16_nd(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                    const uint32_t* box) {
  return encode_tiled_nd(map, false, base, rank, dims, strides, box, true);
}

// [d2][d1][d0] bf16 with row pitch `pitch` (elements), box b0 x b1.
bool map3(CUtensorMap* m, const void* base, int64_t d0, int64_t d1, int64_t d2, int64_t pitch, uint32_t b1) {
  const uint64_t dims[3] = {static_cast<uint64_t>(d0), static_cast<uint64_t>(d1), static_cast<uint64_t>(d2)};
  const uint64_t st[2] = {static_cast<uint64_t>(pitch * 2), static_cast<uint64_t>(pitch * d1 * 2)};
  const uint32_t box[3] = {64, b1, 1};
  return encode_bf16_nd(m, base, 3, dims, st, box);
}
bool map2(CUtensorMap* m, const void* base, int64_t d0, int64_t d1, int64_t pitch, uint32_t b1) {
  const uint64_t dims[2] = {static_cast<uint64_t>(d0), static_cast<uint64_t>(d1)};
  const uint64_t st[1] = {static_cast<uint64_t>(pitch * 2)};
  const uint32_t box[2] = {64, b1};
  return encode_bf16_nd(m, base, 2, dims, st, box);
}
// Token rows, in boxes of 128 and of 32.
bool map_rows(ExGemmParams* p, const void* base, int64_t d0, int64_t rows, int64_t pitch) {
  return map2(&p->mapB, base, d0, rows, pitch, 128 / p->pairs) && map2(&p->mapB32, base, d0, rows, pitch, 32);
}
// A matrix read MN-major in one copy: columns as chunks of 64, box 64 x 64 x chunks.
// `cols` is a multiple of 64; rows of d2 matrices.
bool map_mn(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t pitch, int64_t d2,
            uint32_t chunks) {
  const uint64_t dims[4] = {64, static_cast<uint64_t>(rows), static_cast<uint64_t>(cols / 64),
                            static_cast<uint64_t>(d2)};
  const uint64_t st[3] = {static_cast<uint64_t>(pitch * 2), 128, static_cast<uint64_t>(pitch * rows * 2)};
  const uint32_t box[4] = {64, 64, chunks, 1};
  return encode_bf16_nd(m, base, d2 ? 4 : 3, dims, st, box);
}
// MN-major weights [e][rows][cols]: in one copy where the columns are whole chunks.
bool map_weights_mn(ExGemmParams* p, const void* base, int64_t cols, int64_t rows, int64_t pitch) {
  p->a_whole = cols % 64 == 0;
  return p->a_whole ? map_mn(&p->mapA, base, cols, rows, pitch, p->experts, 2)
                    : map3(&p->mapA, base, cols, rows, p->experts, pitch, 64);
}
// W_in as [e][ip / 8][gate, up][8][hidden]: a box of 64 x 8 x 2 x 8 is 128
// rows, 8 gate rows and 8 up rows in turn.
bool map_up(CUtensorMap* m, const void* base, const muon_experts_t* a, const WeightPlan& w) {
  const uint64_t row = static_cast<uint64_t>(w.hp) * 2;
  const uint64_t dims[5] = {static_cast<uint64_t>(a->hidden), 8, 2, static_cast<uint64_t>(w.ip / 8),
                            static_cast<uint64_t>(a->experts)};
  const uint64_t st[4] = {row, row * w.ip, row * 8, row * 2 * w.ip};
  const uint32_t box[5] = {64, 8, 2, 8, 1};
  return encode_bf16_nd(m, base, 5, dims, st, box);
}

int tiles_of(int64_t n, int64_t per) { return static_cast<int>((n + per - 1) / per); }

// Two CTA pairs to a cluster, one M tile each over the same column tile, whose
// halves each pair loads for both: a quarter less is read from the second-level
// cache, which a power-capped GPU turns into clock (2.9 TFLOP over 8 experts:
// 1972 -> 1864 us).  It needs products that the tensor cores bound: 256 rows an
// expert and 16 steps of K (768 columns, 12 steps: 1172 -> 1176), and M tiles
// that pair up but for one in nine.  Such clusters fit on 144 of 152 SMs, so
// what waits for memory is better off without (48 tokens over 256 experts:
// 233 -> 244).
int pairs_for(const muon_experts_t* a, int64_t rows, int64_t m_rows, int64_t k) {
  const int64_t m_tiles = tiles_of(m_rows, kExMTile);
  return rows >= int64_t{256} * a->experts && k >= 1024 && (m_tiles % 2 == 0 || m_tiles >= 9) ? 2 : 1;
}

ExGemmParams gemm_params(const muon_experts_t* a, const WeightPlan& w, const ApiDevice& d, int pad, int64_t prows,
                         int64_t m_rows, int pairs) {
  ExGemmParams p;
  std::memset(&p, 0, sizeof(p));
  p.offsets = a->offsets;
  p.rows = a->tokens * a->top_k, p.prows = prows;
  p.experts = a->experts;
  p.pad = pad;
  p.pairs = pairs;
  p.m_tiles = tiles_of(m_rows, kExMTile * pairs);
  p.inner = static_cast<int>(a->inner), p.ip = static_cast<int>(w.ip);
  p.ap = p.ip, p.gp = 2 * p.ip;
  p.status = d.status, p.timeout_ns = d.timeout_ns;
  return p;
}

ExSpreadParams spread_params(const muon_experts_t* a, const WeightPlan& w, const ApiDevice& d, int pad,
                             int64_t prows) {
  ExSpreadParams g;
  std::memset(&g, 0, sizeof(g));
  g.x = static_cast<const __nv_bfloat16*>(a->x), g.xs = a->x_stride;
  g.offsets = a->offsets, g.pos = a->pos;
  g.tokens = a->tokens, g.rows = a->tokens * a->top_k, g.hidden = a->hidden, g.hp = w.hp;
  g.experts = a->experts, g.top_k = a->top_k, g.pad = pad;
  g.prows = prows, g.status = d.status;
  return g;
}

ExCombineParams combine_params(const muon_experts_t* a, const ExGemmParams& g, const float* weights,
                               const View& out) {
  ExCombineParams p;
  std::memset(&p, 0, sizeof(p));
  p.y = g.y, p.yp = g.yp, p.yexp = g.yexp, p.yep = g.yep, p.pos = a->pos, p.weights = weights;
  p.out = static_cast<__nv_bfloat16*>(const_cast<void*>(out.p));
  p.outs = out.stride, p.tokens = a->tokens, p.hidden = a->hidden, p.rows = a->tokens * a->top_k;
  p.top_k = a->top_k;
  p.vec = out.rows16();
  return p;
}

// The rows that are summed over slots: 16-bit values, an exponent per 32.
struct RowPlan {
  int64_t yp, yep;
  size_t at_y, at_e;
  RowPlan(int64_t rows, int64_t hidden, Carve* c) : yp(rup(hidden, 8)), yep(rup(hidden, 256) / 32) {
    at_y = c->take(rows * yp * 2);
    at_e = c->take(rows * yep);
  }
  void set(ExGemmParams* p, char* ws) const {
    p->y = reinterpret_cast<__half*>(ws + at_y), p->yp = yp;
    p->yexp = reinterpret_cast<uint8_t*>(ws + at_e), p->yep = yep;
  }
};

// Whether the matrix-vector kernels take a call.  They save the tile kernels'
// launches, copy and sum, about 12 us, but read an expert's weights once for each
// of its rows.  The host does not know the counts: it takes the experts that a
// uniform routing hits on average, and up to 64 MB read twice, which is 11 us.
// Matrix-vector against tiles, us: one token through 8 of 256 x [768, 2048] 23 / 37,
// four 67 / 70; 2 of 8 x [768, 2048], 4 tokens 23 / 30, 8 tokens 39 / 31, 16 tokens
// 67 / 31; 2 of 8 x [14336, 4096], one token 134 / 156, two 254 / 214, 16 tokens
// 1824 / 444; 32 rows of one [512, 1024] 42 / 24, 16 rows 23 / 24.
bool few_rows(const muon_experts_t* a) {
  const int64_t rows = a->tokens * a->top_k;
  if (rows > kExFewRows) return false;
  const double share = std::min(1.0, static_cast<double>(a->top_k) / a->experts);
  const double hit = a->experts * (1.0 - std::pow(1.0 - share, static_cast<double>(a->tokens)));
  return (rows - hit) * 6.0 * static_cast<double>(a->hidden) * static_cast<double>(a->inner) <= 64e6;
}

constexpr int64_t kEarlyRows = 4096;  // most rows whose launches depend early: see launch_after
constexpr int kSpreadBlocks = 5;      // per SM, for a copy that runs alone

muon_status_t experts_impl(const muon_experts_t* a, void* out, int64_t outs, void* gu, cudaStream_t stream) {
  ExpertsViews v;
  bool empty = false;
  MUON_TRY(check_experts(a, &v, &empty));
  if (empty) {
    api_set_launches(0);
    return MUON_OK;
  }
  const int64_t rows = a->tokens * a->top_k, H = a->hidden, I = a->inner;
  const View o{out, MUON_BF16, a->tokens, H, outs}, og = dense(gu, MUON_BF16, rows * 2 * I);
  if (!out || o.bad_stride() || !aligned(out, 2) || !aligned(gu, 2)) return MUON_ERR_INVALID_ARGUMENT;
  if (experts_alias(v, {}, {o, og})) return MUON_ERR_ALIAS;
  std::lock_guard<std::mutex> lock(api_mutex());
  ApiDevice d;
  MUON_TRY(device(&d));
  Carve cv;
  Counter c;
  if (few_rows(a)) {
    const int64_t ip = rup(I, 8);
    const size_t at = cv.take(rows * ip * 4);
    MUON_TRY(cv.open(stream));
    ExFewParams p;
    std::memset(&p, 0, sizeof(p));
    p.x = static_cast<const __nv_bfloat16*>(a->x), p.xs = a->x_stride;
    p.w_in = static_cast<const __nv_bfloat16*>(a->w_in), p.w_out = static_cast<const __nv_bfloat16*>(a->w_out);
    p.weights = a->weights, p.offsets = a->offsets, p.src = a->src, p.pos = a->pos;
    p.gu = static_cast<__nv_bfloat16*>(gu), p.act = reinterpret_cast<float*>(cv.ws + at);
    p.out = static_cast<__nv_bfloat16*>(out), p.outs = outs;
    p.tokens = a->tokens, p.ip = ip, p.rows = static_cast<int>(rows);
    p.hidden = static_cast<int>(H), p.inner = static_cast<int>(I), p.experts = a->experts, p.top_k = a->top_k;
    p.vec_in = v.x.rows16() && aligned(a->w_in, 16) && H % 8 == 0;
    p.vec_out = aligned(a->w_out, 16) && I % 8 == 0;
    p.status = d.status;
    MUON_TRY(c.run(launch_ex_few(p, stream)));
    MUON_TRY(cv.close(stream));
    api_set_launches(2);
    return MUON_OK;
  }
  const WeightPlan w(a, &cv);
  const RowPlan rp(rows, H, &cv);
  const size_t at_x = cv.take(rows * w.hp * 2), at_act = cv.take(rows * w.ip * 2);
  MUON_TRY(cv.open(stream));
  char* const ws = cv.ws;
  __nv_bfloat16* xp = reinterpret_cast<__nv_bfloat16*>(ws + at_x);
  __nv_bfloat16* act = reinterpret_cast<__nv_bfloat16*>(ws + at_act);
  const __nv_bfloat16 *w_in, *w_out;
  MUON_TRY(pack_weights(a, w, ws, &w_in, &w_out, &c, stream));
  const bool early = rows <= kEarlyRows;
  ExSpreadParams g = spread_params(a, w, d, 1, rows);
  g.out = xp;
  g.vec = v.x.rows16();
  MUON_TRY(c.run(launch_ex_spread(g, kSpreadBlocks * d.sms, stream)));
  ExGemmParams up = gemm_params(a, w, d, 1, rows, 2 * w.ip, pairs_for(a, rows, 2 * w.ip, H));
  up.kb = tiles_of(H, 64), up.m = up.inner;
  up.act = act;
  up.gu = static_cast<__nv_bfloat16*>(gu);
  up.gu_vec = aligned(gu, 16) && I % 8 == 0;
  ExGemmParams down = gemm_params(a, w, d, 1, rows, H, pairs_for(a, rows, H, I));
  down.kb = tiles_of(I, 64), down.m = static_cast<int>(H);
  rp.set(&down, ws);
  if (!map_up(&up.mapA, w_in, a, w) || !map_rows(&up, xp, H, rows, w.hp) ||
      !map3(&down.mapA, w_out, I, H, a->experts, w.ip, 128) || !map_rows(&down, act, I, rows, w.ip))
    return MUON_ERR_CUDA;
  MUON_TRY(c.run(launch_ex_gemm(kExUp, up, d.sms, early, stream)));
  MUON_TRY(c.run(launch_ex_gemm(kExDown, down, d.sms, early, stream)));
  MUON_TRY(c.run(launch_ex_combine(combine_params(a, down, a->weights, o), d.sms, early, stream)));
  MUON_TRY(cv.close(stream));
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
  const int64_t rows = a->tokens * a->top_k, H = a->hidden, I = a->inner, per = I * H;
  const View vd{dout, MUON_BF16, a->tokens, H, dos}, vg = dense(gu, MUON_BF16, rows * 2 * I),
             ox{dx, MUON_BF16, a->tokens, H, dxs}, oi = dense(dw_in, dw_dt, 2 * per * a->experts),
             oo = dense(dw_out, dw_dt, per * a->experts), ow = dense(dweights, MUON_F32, rows);
  for (const View* o : {&vd, &vg, &ox, &oi, &oo, &ow})
    if (o->p && (o->bad_stride() || !aligned(o->p, esize(o->dt)))) return MUON_ERR_INVALID_ARGUMENT;
  if (!empty && (!dout || !gu)) return MUON_ERR_INVALID_ARGUMENT;
  if (experts_alias(v, {vd, vg}, {ox, oi, oo, ow})) return MUON_ERR_ALIAS;
  if (empty) {   // no rows: zero weight gradients
    for (const View* o : {&oi, &oo})
      if (o->p && cudaMemsetAsync(const_cast<void*>(o->p), 0, static_cast<size_t>(o->cols * esize(o->dt)),
                                  stream) != cudaSuccess)
        return MUON_ERR_CUDA;
    api_set_launches(0);
    return MUON_OK;
  }
  std::lock_guard<std::mutex> lock(api_mutex());
  ApiDevice d;
  MUON_TRY(device(&d));
  Carve cv;
  const WeightPlan w(a, &cv);
  const RowPlan rp(dx ? rows : 0, H, &cv);
  // padded rows: every expert with rows adds at most kExSeg - 1
  const int64_t prows = rows + (kExSeg - 1) * std::min<int64_t>(a->experts, rows);
  const int parts = tiles_of(I, 128) * 4;
  // pitches of whole 64-column chunks (map_mn); the columns past the data
  // reach only results that are not stored
  const int64_t xpitch = rup(H, 64), gpitch = rup(2 * w.ip, 64), apitch = rup(w.ip, 64);
  const size_t at_x = cv.take(prows * xpitch * 2), at_d = cv.take(prows * xpitch * 2), at_wr = cv.take(prows * 4),
               at_dgu = cv.take(prows * gpitch * 2), at_wa = cv.take(prows * apitch * 2),
               at_part = cv.take(rows * parts * 4);
  MUON_TRY(cv.open(stream));
  char* const ws = cv.ws;
  __nv_bfloat16* xp = reinterpret_cast<__nv_bfloat16*>(ws + at_x);
  __nv_bfloat16* dop = reinterpret_cast<__nv_bfloat16*>(ws + at_d);
  __nv_bfloat16* dgu = reinterpret_cast<__nv_bfloat16*>(ws + at_dgu);
  __nv_bfloat16* wact = reinterpret_cast<__nv_bfloat16*>(ws + at_wa);
  Counter c;
  const __nv_bfloat16 *w_in, *w_out;
  MUON_TRY(pack_weights(a, w, ws, &w_in, &w_out, &c, stream));
  ExSpreadParams g = spread_params(a, w, d, kExSeg, prows);
  g.hp = xpitch;
  g.x = static_cast<const __nv_bfloat16*>(dout), g.xs = dos, g.out = dop;
  g.vec = vd.rows16();
  g.weights = a->weights;
  g.wr = reinterpret_cast<float*>(ws + at_wr);
  MUON_TRY(c.run(launch_ex_spread(g, kSpreadBlocks * d.sms, stream)));
  // x's rows, for dw_in, are copied beside something: with many rows while dx's
  // product runs (the copy needs HBM, the product the tensor cores; one block an
  // SM leaves it room), else while dout's are.  8192 tokens over 64 experts of
  // [768, 2048]: 1094 -> 1080 us.  Cutting the forward's copy and first product
  // in two to do the same: 1104 -> 1114 us on 16384 tokens over 256.
  const bool many = rows >= 16384, beside = dx && dw_in && many;
  const bool early = rows <= kEarlyRows;
  auto copy_x = [&](int blocks, bool with_previous) {
    g.x = static_cast<const __nv_bfloat16*>(a->x), g.xs = a->x_stride, g.out = xp;
    g.vec = v.x.rows16();
    g.wr = nullptr;
    g.beside = with_previous;
    return c.run(launch_ex_spread(g, blocks * d.sms, stream));
  };
  float* const wr = g.wr;
  if (dw_in && !beside) MUON_TRY(copy_x(kSpreadBlocks, true));
  ExGemmParams da = gemm_params(a, w, d, kExSeg, prows, I, 1);
  da.kb = tiles_of(H, 64), da.m = da.inner;
  da.gu = static_cast<__nv_bfloat16*>(const_cast<void*>(gu));
  da.gu_vec = aligned(gu, 16) && I % 8 == 0;
  da.wr = wr, da.dgu = dgu, da.act = wact;
  da.ap = static_cast<int>(apitch), da.gp = static_cast<int>(gpitch);
  da.part = reinterpret_cast<float*>(ws + at_part);
  if (!map_weights_mn(&da, w_out, I, H, w.ip) || !map_rows(&da, dop, H, prows, xpitch))
    return MUON_ERR_CUDA;
  MUON_TRY(c.run(launch_ex_gemm(kExDact, da, d.sms, early, stream)));
  if (dweights) {
    const ExWeightParams wp{da.part, a->pos, dweights, rows, parts};
    MUON_TRY(c.run(launch_ex_dweights(wp, early, stream)));
  }
  if (beside) MUON_TRY(copy_x(1, false));
  if (dx) {
    ExGemmParams p = gemm_params(a, w, d, kExSeg, prows, H, pairs_for(a, prows, H, 2 * I));
    p.beside = beside;
    p.kb = tiles_of(2 * w.ip, 64), p.m = static_cast<int>(H);
    rp.set(&p, ws);
    if (!map_weights_mn(&p, w_in, H, 2 * w.ip, w.hp) || !map_rows(&p, dgu, 2 * w.ip, prows, gpitch))
      return MUON_ERR_CUDA;
    MUON_TRY(c.run(launch_ex_gemm(kExDx, p, d.sms, beside || early, stream)));
    MUON_TRY(c.run(launch_ex_combine(combine_params(a, p, nullptr, ox), d.sms, early, stream)));
  }
  for (int k = 0; k < 2; ++k) {
    void* out = k ? dw_out : dw_in;
    if (!out) continue;
    const int64_t m = k ? H : 2 * w.ip;
    ExGemmParams p = gemm_params(a, w, d, kExSeg, prows, m, pairs_for(a, prows, m, prows / a->experts));
    p.m = static_cast<int>(m), p.n = static_cast<int>(k ? I : H);
    p.n_tiles = tiles_of(p.n, kExNTile);
    p.dw = out, p.dw_dt = dw_dt;
    p.dw_vec = aligned(out, 16) && p.n * esize(dw_dt) % 16 == 0;
    const int64_t ap = k ? xpitch : gpitch, bp = k ? apitch : xpitch;
    if (!map_mn(&p.mapA, k ? dop : dgu, ap, prows, ap, 0, 2) ||
        !map_mn(&p.mapB, k ? wact : xp, bp, prows, bp, 0, 2 / p.pairs))
      return MUON_ERR_CUDA;
    MUON_TRY(c.run(launch_ex_gemm(k ? kExDwOut : kExDwIn, p, d.sms, early, stream)));
  }
  MUON_TRY(cv.close(stream));
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
