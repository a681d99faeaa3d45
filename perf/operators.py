"""The operators of a mixture-of-experts block that are timed and compared.

Three operators, each with its gradient, as a training or serving program calls
them between the optimizer's steps:

  norm     h = x + residual, y = gain * h / sqrt(mean(h^2) + eps), with y in
           f32, bf16 or as e4m3 codes with f32 scales; and its gradient.
  route    scores of the experts from logits, a balance bias that only the
           choice sees, expert groups, top-k, renormalised weights, and the
           list of (token, slot) rows in expert order; and its gradient.
  experts  out[t] = sum_j w[t,j] W_out[e] (silu(W_gate[e] x_t) * (W_up[e] x_t)),
           e = idx[t,j], with w_in[e] = (W_gate[e]; W_up[e]); and its gradient.

`own` false computes them from elementary torch operations in 32 bits, rounded
once at the end; `own` true calls the library.  `exact` computes them in 64 bits
from the definitions.
"""
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0
SCALE_FLOOR = 1e-12      # the least largest magnitude that an e4m3 scale stands for
EPS = 1e-6
BIAS_UNIT = 2.0 ** -10   # step of the balance bias


# ---- cases --------------------------------------------------------------------------
def listed():
    return [
        # one token of a decode step: launch latency
        dict(name="norm token", op="norm", back=False, rows=1, cols=4096, x="bf16", res="bf16",
             out="bf16", group=0),
        # a ragged prompt into 8-bit projections, f32 residual stream
        dict(name="norm prompt e4m3", op="norm", back=False, rows=4099, cols=2048, x="bf16",
             res="f32", out="e4m3", group=128),
        # a training micro-batch of the widest model dimension
        dict(name="norm batch", op="norm", back=False, rows=16384, cols=8192, x="bf16",
             res="bf16", out="bf16", group=0),
        # its gradient at the Llama-3-8B width, with the residual stream's gradient
        dict(name="norm batch gradient", op="norm", back=True, rows=16384, cols=4096, x="bf16",
             res="bf16", out="bf16", group=0),
        # a decode step of 48 sequences over 256 experts in groups
        dict(name="route decode", op="route", back=False, tokens=48, experts=256, top_k=8,
             score="sigmoid", bias=True, groups=8, top_groups=4, group_score="sum2",
             renorm=True, scale=2.5, logits="f32", keep=1.0),
        # a training batch over 256 experts, one token in 16 padding
        dict(name="route batch", op="route", back=False, tokens=16384, experts=256, top_k=8,
             score="sigmoid", bias=True, groups=8, top_groups=4, group_score="sum2",
             renorm=True, scale=2.5, logits="f32", keep=0.9375),
        # gradient of a softmax router without renormalisation, an odd batch
        dict(name="route gradient", op="route", back=True, tokens=16381, experts=128, top_k=8,
             score="softmax", bias=False, groups=1, top_groups=1, group_score="max",
             renorm=False, scale=1.0, logits="bf16", keep=1.0),
        # one token through 8 of 256 experts of [768, 2048]: 75 MB of weights
        dict(name="experts token", op="experts", back=False, tokens=1, experts=256, top_k=8,
             hidden=2048, inner=768, save=False, keep=1.0),
        # a decode step of 48 sequences: nearly every expert, one or two rows each
        dict(name="experts decode", op="experts", back=False, tokens=48, experts=256, top_k=8,
             hidden=2048, inner=768, save=False, keep=1.0),
        # a ragged prompt through 8 experts of the Llama-3-8B feed-forward shape
        dict(name="experts prompt wide", op="experts", back=False, tokens=4093, experts=8,
             top_k=2, hidden=4096, inner=14336, save=False, keep=1.0),
        # a training batch through 256 experts, one token in 16 padding
        dict(name="experts batch", op="experts", back=False, tokens=16384, experts=256, top_k=8,
             hidden=2048, inner=768, save=True, keep=0.9375),
        # the gradient over 64 experts
        dict(name="experts gradient", op="experts", back=True, tokens=8192, experts=64, top_k=8,
             hidden=2048, inner=768, save=True, keep=1.0),
    ]


def draw(rng):
    """One more case of the same ranges; sizes spread over their logarithm."""
    def size(lo, hi):
        n = min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))
        return n + 1 if n in (1536, 3072) else n

    def width(lo, hi):    # mostly multiples of 64 or 8, one in eight of any value
        unit = rng.choice((64, 64, 64, 8, 8, 8, 8, 1))
        n = max(unit, size(lo, hi) // unit * unit)
        return n + unit if n in (1536, 3072) else n

    op = rng.choice(("norm", "route", "experts", "experts"))
    back = rng.random() < 0.4
    if op == "norm":
        while True:
            rows, cols = size(1, 32768), width(64, 16384)
            if rows * cols <= (1 << 26 if back else 1 << 27):
                break
        out = "bf16" if back else rng.choice(("bf16", "f32", "e4m3"))
        return dict(op=op, back=back, rows=rows, cols=cols, x=rng.choice(("bf16", "bf16", "f32")),
                    res=rng.choice(("bf16", "f32", "none")), out=out,
                    group=rng.choice((0, 128)) if out == "e4m3" else 0)
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * size(4, 320 // groups)
        top_groups = rng.randint(max(1, groups // 2), groups)
        top_k = min(size(1, 16), experts // groups * top_groups)
        # a softmax router's groups go by their best expert, without a bias
        score = rng.choice(("sigmoid", "softmax"))
        return dict(op=op, back=back, tokens=size(1, 16384), experts=experts, top_k=top_k,
                    score=score, bias=score == "sigmoid" and rng.random() < 0.7, groups=groups,
                    top_groups=top_groups,
                    group_score=rng.choice(("sum2", "max")) if score == "sigmoid" else "max",
                    renorm=rng.random() < 0.5, scale=rng.choice((1.0, 2.5)),
                    logits=rng.choice(("f32", "bf16")), keep=rng.choice((1.0, 0.9)))
    while True:
        experts = size(4, 256)
        top_k = min(size(1, 8), experts)
        tokens, hidden, inner = size(1, 16384), width(128, 4096), width(64, 4096)
        weights = experts * hidden * inner
        if weights <= (64 if back else 256) * 2048 * 768 and \
                tokens * top_k * hidden * inner <= (65536 if back else 131072) * 2048 * 768:
            break
    return dict(op=op, back=back, tokens=tokens, experts=experts, top_k=top_k, hidden=hidden,
                inner=inner, save=back or rng.random() < 0.5, keep=rng.choice((1.0, 0.9)))


# ---- inputs -------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(gen, *shape, dtype=torch.float32, scale=1.0):
    t = torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)
    return t.mul_(scale) if scale != 1.0 else t


def _mask(gen, tokens, keep):
    if keep >= 1.0:
        return None
    order = torch.randperm(tokens, generator=gen, device="cuda")
    return order < max(1, round(keep * tokens))


def prepare(case, seed):
    gen = _generator(seed)
    s = dict(case=case)
    if case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        # a few columns carry large values, as hidden states do
        spread = 1.0 + 9.0 * (torch.rand(cols, generator=gen, device="cuda") < 0.01)
        s["gain"] = (1.0 + _randn(gen, cols, scale=0.1)).to(torch.bfloat16)
        x, res = DTYPES[case["x"]], case["res"]
        if case["back"]:
            s["h"] = (_randn(gen, rows, cols) * spread).to(x)
            s["dy"] = _randn(gen, rows, cols, dtype=x)
            s["dres"] = None if res == "none" else _randn(gen, rows, cols, dtype=DTYPES[res])
        else:
            s["x"] = _randn(gen, rows, cols, dtype=x)
            s["res"] = None if res == "none" else (_randn(gen, rows, cols) * spread).to(DTYPES[res])
        return s
    tokens, experts, k = case["tokens"], case["experts"], case["top_k"]
    # some experts are more popular than others
    logits = _randn(gen, tokens, experts) + _randn(gen, experts, scale=0.5)
    mask = _mask(gen, tokens, case["keep"])
    if case["op"] == "route":
        s["logits"] = logits.to(DTYPES[case["logits"]])
        s["mask"] = mask
        s["bias"] = None
        if case["bias"]:
            s["bias"] = BIAS_UNIT * torch.randint(-64, 65, (experts,), generator=gen,
                                                  device="cuda").float()
        if case["back"]:
            s["idx"] = _route(s)[0]
            s["dweights"] = _randn(gen, tokens, k)
        return s
    # a routing that a router has made: choice, weights and row order
    top = logits.topk(k, dim=1)
    idx = top.indices
    if mask is not None:
        idx = torch.where(mask[:, None], idx, -1)
    s["weights"] = torch.where(idx >= 0, top.values.softmax(1), 0.0)
    s["idx"] = idx.to(torch.int32)
    s["offsets"], s["src"], s["pos"] = _plan(s["idx"], experts)
    s["n_rows"] = int(s["offsets"][-1])
    s["cap"] = int(s["offsets"].diff().max())
    hidden, inner = case["hidden"], case["inner"]
    s["x"] = _randn(gen, tokens, hidden, dtype=torch.bfloat16)
    s["w_in"] = _randn(gen, experts, 2 * inner, hidden, dtype=torch.bfloat16, scale=hidden ** -0.5)
    s["w_out"] = _randn(gen, experts, hidden, inner, dtype=torch.bfloat16, scale=inner ** -0.5)
    if case["back"]:
        s["dout"] = _randn(gen, tokens, hidden, dtype=torch.bfloat16)
        # what a forward pass has saved: gate and up rows before the activation
        s["gu"] = torch.empty(tokens * k, 2 * inner, dtype=torch.bfloat16, device="cuda")
        ends = s["offsets"].tolist()
        token = s["src"].long() // k
        for e in range(experts):
            a, b = ends[e], ends[e + 1]
            if b > a:
                s["gu"][a:b] = s["x"][token[a:b]] @ s["w_in"][e].t()
        s["gu"][s["n_rows"]:] = 0
    return s


# ---- plain forms --------------------------------------------------------------------
def _norm(s):
    c = s["case"]
    x = s["x"].float()
    h = x if s["res"] is None else x + s["res"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["gain"].float()
    out = {} if s["res"] is None else {"h": h.to(s["res"].dtype)}
    if c["out"] != "e4m3":
        out["y"] = y.to(DTYPES[c["out"]])
        return out
    group = c["group"] or c["cols"]
    n = -(-c["cols"] // group)
    padded = torch.nn.functional.pad(y, (0, n * group - c["cols"])).view(-1, n, group)
    top = padded.abs().amax(2, keepdim=True).clamp(min=SCALE_FLOOR)
    codes = (padded * (E4M3_MAX / top)).clamp(-E4M3_MAX, E4M3_MAX)
    out["y"] = codes.view(-1, n * group)[:, :c["cols"]].to(torch.float8_e4m3fn)
    out["scales"] = (top / E4M3_MAX).squeeze(2)
    return out


def _norm_gradient(s):
    h, dy = s["h"].float(), s["dy"].float()
    rstd = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    unit = h * rstd
    g = dy * s["gain"].float()
    dh = rstd * (g - unit * (g * unit).mean(1, keepdim=True))
    if s["dres"] is not None:
        dh = dh + s["dres"].float()
    return {"dh": dh.to(s["h"].dtype), "dgain": (dy * unit).sum(0)}


def _plan(idx, experts):
    """Rows (token * k + slot) in expert order: offsets, src by row, row by (token, slot)."""
    n = idx.numel()
    e = torch.where(idx >= 0, idx, experts).reshape(-1).long()
    counts = torch.zeros(experts + 1, dtype=torch.int32, device=idx.device)
    counts.scatter_add_(0, e, torch.ones(n, dtype=torch.int32, device=idx.device))
    ends = counts.cumsum(0)
    offsets = (ends - counts).to(torch.int32)
    order = torch.sort(e, stable=True).indices
    row = torch.arange(n, device=idx.device)
    live = row < offsets[experts]
    src = torch.where(live, order, -1).to(torch.int32)
    pos = torch.empty(n, dtype=torch.int32, device=idx.device)
    pos[order] = torch.where(live, row, -1).to(torch.int32)
    return offsets, src, pos.view(idx.shape)


def _scores(s):
    x = s["logits"].float()
    x = torch.where(torch.isfinite(x), x, float("-inf"))
    if s["case"]["score"] == "sigmoid":
        return x, torch.reciprocal(1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True).clamp(min=torch.finfo(torch.float32).min))
    return x, e / e.sum(1, keepdim=True).clamp(min=1.0)    # the largest term is 1


def _route(s):
    c = s["case"]
    experts, k = c["experts"], c["top_k"]
    x, score = _scores(s)
    # both scores grow with the logit: without a bias the choice goes by the logit;
    # an expert whose logit is not finite is never chosen
    dead = torch.isinf(x)
    key = x if s["bias"] is None else torch.where(dead, x, score + s["bias"])
    if c["groups"] > 1:
        per = experts // c["groups"]
        grouped = key.view(-1, c["groups"], per)
        if c["group_score"] == "sum2":
            both = torch.where(dead, x, score) if s["bias"] is None else key
            two = torch.sort(both.view(-1, c["groups"], per), dim=2, descending=True).values[:, :, :2]
            best = torch.where(torch.isinf(two[:, :, 0]), two[:, :, 0],
                               torch.where(torch.isinf(two), 0.0, two).sum(2))
        else:
            best = grouped.amax(2)
        chosen = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        allowed = torch.zeros_like(best, dtype=torch.bool).scatter_(1, chosen, True)
        key = torch.where(allowed[:, :, None], grouped, float("-inf")).view(-1, experts)
    ranked = torch.sort(key, dim=1, descending=True, stable=True)
    idx = torch.where(torch.isinf(ranked.values), -1, ranked.indices)[:, :k]
    if s["mask"] is not None:
        idx = torch.where(s["mask"][:, None], idx, -1)
    w = torch.where(idx >= 0, score.gather(1, idx.clamp(min=0)), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return idx.to(torch.int32), w * c["scale"]


def _route_gradient(s):
    c = s["case"]
    _, score = _scores(s)
    live = s["idx"] >= 0
    at = s["idx"].long().clamp(min=0)
    d = torch.where(live, s["dweights"] * c["scale"], 0.0)
    q = torch.where(live, score.gather(1, at), 0.0)
    if c["renorm"]:
        total = q.sum(1, keepdim=True)
        share = torch.where(total > 0, q / total, 0.0)
        d = torch.where(total > 0, (d - (d * share).sum(1, keepdim=True)) / total, 0.0)
    if c["score"] == "sigmoid":
        grad = torch.zeros_like(score).scatter_add_(1, at, d * q * (1.0 - q))
    else:
        grad = torch.zeros_like(score).scatter_add_(1, at, d * q)
        if not c["renorm"]:
            grad = grad - score * (d * q).sum(1, keepdim=True)
    return grad.to(s["logits"].dtype)


def _padded(s):
    """Expert and place of every row, and a token's rows as [experts, cap, width]."""
    src = s["src"][:s["n_rows"]].long()
    e = s["idx"].reshape(-1)[src].long()
    place = torch.arange(s["n_rows"], device=src.device) - s["offsets"][e].long()

    def spread(rows):
        out = torch.zeros(s["case"]["experts"], s["cap"], rows.shape[1], device=rows.device)
        out[e, place] = rows
        return out

    return src, src // s["case"]["top_k"], e, place, spread


def _sum_slots(s, rows, weights):
    live = s["pos"] >= 0
    picked = rows[s["pos"].long().clamp(min=0)]
    w = torch.where(live, weights, 0.0) if weights is not None else live.float()
    return (picked * w[:, :, None]).sum(1)


def _experts(s):
    c = s["case"]
    _, token, e, place, spread = _padded(s)
    gu = torch.bmm(spread(s["x"].float()[token]), s["w_in"].float().transpose(1, 2))
    gate, up = gu.chunk(2, dim=2)
    act = gate / (1.0 + torch.exp(-gate)) * up
    y = torch.bmm(act, s["w_out"].float().transpose(1, 2))[e, place]
    out = {"out": _sum_slots(s, y, s["weights"]).to(torch.bfloat16)}
    if c["save"]:
        out["gu"] = gu[e, place].to(torch.bfloat16)
    return out


def _experts_gradient(s):
    src, token, e, place, spread = _padded(s)
    gate, up = s["gu"][:s["n_rows"]].float().chunk(2, dim=1)
    sig = 1.0 / (1.0 + torch.exp(-gate))
    act = gate * sig * up
    dout = spread(s["dout"].float()[token])
    dact = torch.bmm(dout, s["w_out"].float())[e, place]
    w = s["weights"].reshape(-1)[src][:, None]
    dweights = torch.zeros(s["weights"].numel(), device=src.device)
    dweights[src] = (dact * act).sum(1)
    dact = dact * w
    dgu = spread(torch.cat((dact * up * sig * (1.0 + gate * (1.0 - sig)), dact * gate * sig), 1))
    dx = torch.bmm(dgu, s["w_in"].float())[e, place]
    dw_in = torch.bmm(dgu.transpose(1, 2), spread(s["x"].float()[token]))
    dw_out = torch.bmm(dout.transpose(1, 2), spread(act * w))
    return {"dx": _sum_slots(s, dx, None).to(torch.bfloat16), "dw_in": dw_in.to(torch.bfloat16),
            "dw_out": dw_out.to(torch.bfloat16), "dweights": dweights.view_as(s["weights"])}


# ---- the library's calls ------------------------------------------------------------
def _call(s):
    from newton_schulz_gb300 import binding as B
    c = s["case"]
    if c["op"] == "norm":
        if c["back"]:
            dh, dgain = B.muon_rmsnorm_backward(s["dy"], s["h"], s["gain"], dres=s["dres"], eps=EPS)
            return {"dh": dh, "dgain": dgain}
        y, h, scales = B.muon_rmsnorm_forward(s["x"], s["gain"], residual=s["res"], eps=EPS,
                                              y_dtype=DTYPES[c["out"]], group=c["group"])
        out = {"y": y}
        if h is not None:
            out["h"] = h
        if scales is not None:
            out["scales"] = scales
        return out
    if c["op"] == "route":
        cfg = B.make_route_config(
            c["experts"], c["top_k"],
            score=B.ROUTE_SIGMOID if c["score"] == "sigmoid" else B.ROUTE_SOFTMAX,
            groups=c["groups"], top_groups=c["top_groups"],
            group_score=B.GROUP_SUM2 if c["group_score"] == "sum2" else B.GROUP_MAX,
            renormalize=c["renorm"], scale=c["scale"])
        if c["back"]:
            return B.muon_route_backward(s["logits"], cfg, s["idx"], s["dweights"])
        r = B.muon_route_forward(s["logits"], cfg, bias=s["bias"], mask=s["mask"])
        return list(r)
    r = B.Route(s["idx"], s["weights"], s["offsets"], s["src"], s["pos"])
    if c["back"]:
        dx, dw_in, dw_out, dweights = B.muon_experts_backward(
            s["dout"], s["x"], s["w_in"], s["w_out"], r, s["gu"], dw_dtype=torch.bfloat16)
        return {"dx": dx, "dw_in": dw_in, "dw_out": dw_out, "dweights": dweights}
    out, gu = B.muon_experts_forward(s["x"], s["w_in"], s["w_out"], r, save=c["save"])
    return {"out": out, "gu": gu[:s["n_rows"]]} if c["save"] else {"out": out}


def run(state):
    if own:
        return _call(state)
    c = state["case"]
    if c["op"] == "norm":
        return _norm_gradient(state) if c["back"] else _norm(state)
    if c["op"] == "route":
        if c["back"]:
            return _route_gradient(state)
        idx, w = _route(state)
        return [idx, w, *_plan(idx, c["experts"])]
    return _experts_gradient(state) if c["back"] else _experts(state)


# ---- what one pass cannot do without ---------------------------------------------------
def work(case):
    c, wide = case, {"f32": 4, "bf16": 2, "e4m3": 1, "none": 0}
    if c["op"] == "norm":
        n, r = c["rows"] * c["cols"], wide[c["res"]]
        if c["back"]:    # dy and h read, dh written, the residual gradient read
            return {"bytes": n * (3 * wide[c["x"]] + r) + 6 * c["cols"], "flops": 9 * n}
        scales = 4 * c["rows"] * -(-c["cols"] // (c["group"] or c["cols"]))
        return {"bytes": n * (wide[c["x"]] + 2 * r + wide[c["out"]]) + 2 * c["cols"] +
                (scales if c["out"] == "e4m3" else 0), "flops": 5 * n}
    if c["op"] == "route":
        n, picks = c["tokens"] * c["experts"], c["tokens"] * c["top_k"]
        if c["back"]:    # logits read, their gradient written, idx and dweights read
            return {"bytes": 2 * n * wide[c["logits"]] + 8 * picks, "flops": 8 * n}
        # logits read; idx, weights, src and pos written
        return {"bytes": n * wide[c["logits"]] + 16 * picks + 8 * c["experts"], "flops": 8 * n}
    tokens, hidden, inner = c["tokens"], c["hidden"], c["inner"]
    rows = c["keep"] * tokens * c["top_k"]
    hit = c["experts"] * (1.0 - (1.0 - c["top_k"] / c["experts"]) ** (c["keep"] * tokens))
    weights = 2.0 * hit * 3 * hidden * inner
    if c["back"]:    # x, dout, gu and the weights read; dx and every weight's gradient written
        return {"bytes": weights + 2.0 * c["experts"] * 3 * hidden * inner +
                6.0 * tokens * hidden + rows * (4.0 * inner + 8), "flops": 12.0 * rows * hidden * inner}
    return {"bytes": weights + 4.0 * tokens * hidden + rows * 12 + (4.0 * rows * inner if c["save"] else 0),
            "flops": 6.0 * rows * hidden * inner}


# ---- 64 bits ------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    up = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
          for k, v in s.items()}
    return {"norm": _exact_norm, "route": _exact_route, "experts": _exact_experts}[case["op"]](case, s, up)


def _exact_norm(c, s, d):
    n = c["cols"]
    if c["back"]:
        h, dy, w = d["h"], d["dy"], d["gain"]
        ms = h.square().sum(1) / n + EPS
        inner = (dy * w * h).sum(1)
        dh = (dy * w) / ms.sqrt()[:, None] - h * (inner / (n * ms ** 1.5))[:, None]
        if d["dres"] is not None:
            dh += d["dres"]
        return {"dh": dh, "dgain": (dy * h / ms.sqrt()[:, None]).sum(0)}
    h = d["x"].clone()
    if d["res"] is not None:
        h += d["res"]
    y = h / (h.square().sum(1) / n + EPS).sqrt()[:, None] * d["gain"]
    out = {"y": y}
    if d["res"] is not None:
        out["h"] = h
    if c["out"] == "e4m3":
        group = c["group"] or n
        tops = torch.stack([y[:, a:a + group].abs().max(1).values for a in range(0, n, group)], 1)
        tops = tops.clamp(min=SCALE_FLOOR)
        wide = tops.repeat_interleave(group, 1)[:, :n]
        out["y"], out["scales"] = y * E4M3_MAX / wide, tops / E4M3_MAX
    return out


def _exact_route(c, s, d):
    x = d["logits"]
    p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, 1)
    if c["back"]:
        # differentiate the weights' definition
        x = x.clone().requires_grad_(True)
        p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, 1)
        at = s["idx"].long()
        w = p.gather(1, at.clamp(min=0)) * (at >= 0)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        (w * c["scale"] * d["dweights"]).sum().backward()
        return x.grad
    idx = _route(s)[0].long()    # whole numbers: their order is the operator's rule
    w = p.gather(1, idx.clamp(min=0)) * (idx >= 0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return [None, w * c["scale"], None, None, None]


def _exact_experts(c, s, d):
    tokens, k, inner, n = c["tokens"], c["top_k"], c["inner"], s["n_rows"]
    if (12.0 if c["back"] else 6.0) * tokens * k * c["hidden"] * inner > 6e12:    # over some seconds
        return None
    ends = s["offsets"].tolist()
    src = s["src"].long()
    zero = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")  # noqa: E731
    out, gu, dx = zero(tokens, c["hidden"]), zero(n, 2 * inner), zero(tokens, c["hidden"])
    dw = zero(tokens * k)
    if c["back"]:
        dw_in, dw_out = zero(*s["w_in"].shape), zero(*s["w_out"].shape)
    for e in range(c["experts"]):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        t = src[a:b] // k
        w = d["weights"].reshape(-1)[src[a:b], None]
        w_in, w_out = s["w_in"][e].double(), s["w_out"][e].double()
        both = d["gu"][a:b] if c["back"] else d["x"][t] @ w_in.t()
        gate, up = both[:, :inner], both[:, inner:]
        silu = gate * torch.sigmoid(gate)
        act = silu * up
        if not c["back"]:
            gu[a:b] = both
            out.index_add_(0, t, w * (act @ w_out.t()))
            continue
        dact = d["dout"][t] @ w_out
        dw[src[a:b]] = (dact * act).sum(1)
        slope = torch.sigmoid(gate) * (1 + gate * torch.sigmoid(-gate))
        dboth = torch.cat((w * dact * up * slope, w * dact * silu), 1)
        dx.index_add_(0, t, dboth @ w_in)
        dw_in[e] = dboth.t() @ d["x"][t]
        dw_out[e] = d["dout"][t].t() @ (w * act)
    if c["back"]:
        return {"dx": dx, "dw_in": dw_in, "dw_out": dw_out, "dweights": dw.view(tokens, k)}
    return {"out": out, "gu": gu} if c["save"] else {"out": out}
