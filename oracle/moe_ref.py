"""Float64 oracle of the mixture-of-experts block's operators: RMS norm with
the residual's addition, routing and its row plan, the experts' products, and
their gradients.  Plain loops over rows and slots, written from the formulas
in include/muon.h; shares no code with the library."""
import math

import numpy as np


# ---- RMS norm ------------------------------------------------------------------------
def rmsnorm_ref(x, residual, gain, eps):
    x = np.asarray(x, np.float64)
    h = x if residual is None else x + np.asarray(residual, np.float64)
    y = np.empty_like(h)
    for r in range(h.shape[0]):
        rms = math.sqrt(float(np.dot(h[r], h[r])) / h.shape[1] + eps)
        y[r] = h[r] / rms * (1.0 if gain is None else gain)
    return h, y


def e4m3_pieces(y, group):
    """(scaled values before rounding, scales) of rows cut into `group` columns (0: whole rows)."""
    rows, cols = y.shape
    g = group or cols
    n = -(-cols // g)
    scales, codes = np.empty((rows, n)), np.empty_like(y)
    for p in range(n):
        part = y[:, p * g:(p + 1) * g]
        top = np.maximum(np.abs(part).max(1), 1e-12)
        scales[:, p] = top / 448.0
        codes[:, p * g:(p + 1) * g] = part * (448.0 / top)[:, None]
    return codes, scales


def rmsnorm_grad_ref(dy, h, gain, dres, eps):
    dy, h = np.asarray(dy, np.float64), np.asarray(h, np.float64)
    n = h.shape[1]
    dh, dgain = np.empty_like(h), np.zeros(n)
    for r in range(h.shape[0]):
        inv = 1.0 / math.sqrt(float(np.dot(h[r], h[r])) / n + eps)
        u = h[r] * inv
        g = dy[r] if gain is None else dy[r] * gain
        dh[r] = inv * (g - u * (float(np.dot(g, u)) / n))
        dgain += dy[r] * u
    if dres is not None:
        dh += dres
    return dh, dgain


# ---- routing -------------------------------------------------------------------------
def _scores(row, score):
    row = np.where(np.isfinite(row), row, -np.inf)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return row, 1.0 / (1.0 + np.exp(-row))
    top = row.max()
    if top == -np.inf:
        return row, np.zeros_like(row)
    e = np.exp(row - top)
    return row, e / e.sum()


def _best(values, live, count):
    """Indices of the `count` largest live values, ties to the lowest index."""
    order = sorted((i for i in range(len(values)) if live[i]), key=lambda i: (-values[i], i))
    return order[:count]


def route_ref(logits, top_k, score="softmax", bias=None, mask=None, groups=1, top_groups=None,
              group_score="max", renormalize=False, scale=1.0):
    logits = np.asarray(logits, np.float64)
    tokens, experts = logits.shape
    top_groups = groups if top_groups is None else top_groups
    idx = np.full((tokens, top_k), -1, np.int64)
    weights = np.zeros((tokens, top_k))
    per = experts // groups
    for t in range(tokens):
        if mask is not None and not mask[t]:
            continue
        row, s = _scores(logits[t], score)
        live = row > -np.inf
        biased = s if bias is None else s + np.asarray(bias, np.float64)
        key = row if bias is None else biased
        if top_groups < groups:
            rank, alive = np.zeros(groups), np.zeros(groups, bool)
            for g in range(groups):
                mine = [i for i in range(g * per, (g + 1) * per) if live[i]]
                alive[g] = bool(mine)
                if mine and group_score == "max":
                    rank[g] = max(key[i] for i in mine)
                elif mine:
                    rank[g] = sum(sorted((biased[i] for i in mine), reverse=True)[:2])
            kept = set(_best(rank, alive, top_groups))
            live = live & np.array([i // per in kept for i in range(experts)])
        chosen = _best(key, live, top_k)
        idx[t, :len(chosen)] = chosen
        w = s[chosen]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
        weights[t, :len(chosen)] = scale * w
    return idx, weights


def route_weights_ref(logits, idx, score, renormalize, scale):
    """The weights as a function of the logits with the choice held fixed."""
    out = np.zeros(idx.shape)
    for t in range(idx.shape[0]):
        _, s = _scores(np.asarray(logits[t], np.float64), score)
        w = np.array([s[e] if e >= 0 else 0.0 for e in idx[t]])
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
        out[t] = scale * w
    return out


def route_grad_ref(logits, idx, dweights, score, renormalize, scale):
    logits = np.asarray(logits, np.float64)
    grad = np.zeros_like(logits)
    for t in range(logits.shape[0]):
        _, s = _scores(logits[t], score)
        ds = np.zeros_like(s)
        at = [(j, e) for j, e in enumerate(idx[t]) if 0 <= e < len(s)]
        total = sum(s[e] for _, e in at)
        for j, e in at:
            if not renormalize:
                ds[e] += scale * dweights[t, j]
            elif total > 0:
                mean = sum(dweights[t, i] * s[f] for i, f in at) / total
                ds[e] += scale * (dweights[t, j] - mean) / total
        if score == "sigmoid":
            grad[t] = ds * s * (1.0 - s)
        else:
            grad[t] = s * (ds - float(np.dot(ds, s)))
    return grad


def plan_ref(idx, experts):
    idx = np.asarray(idx)
    flat = idx.reshape(-1)
    rows = [i for e in range(experts) for i in range(len(flat)) if flat[i] == e]
    offsets = np.zeros(experts + 1, np.int64)
    for e in range(experts):
        offsets[e + 1] = offsets[e] + int((flat == e).sum())
    src = np.full(len(flat), -1, np.int64)
    pos = np.full(len(flat), -1, np.int64)
    for r, i in enumerate(rows):
        src[r], pos[i] = i, r
    return offsets, src, pos.reshape(idx.shape)


# ---- experts' products ------------------------------------------------------------------
def _parts(gu):
    inner = gu.shape[0] // 2
    g, u = gu[:inner], gu[inner:]
    s = 1.0 / (1.0 + np.exp(-g))
    return g, u, s


def experts_ref(x, w_in, w_out, idx, weights):
    """(out, gu by (token, slot)); slots with idx -1 have zero gu."""
    tokens, k = idx.shape
    out = np.zeros_like(x)
    gu = np.zeros((tokens, k, w_in.shape[1]))
    for t in range(tokens):
        for j in range(k):
            e = idx[t, j]
            if e < 0:
                continue
            gu[t, j] = w_in[e] @ x[t]
            g, u, s = _parts(gu[t, j])
            out[t] += weights[t, j] * (w_out[e] @ (g * s * u))
    return out, gu


def experts_grad_ref(dout, x, w_in, w_out, idx, weights, gu):
    """(dx, dw_in, dw_out, dweights) from the saved gu by (token, slot)."""
    tokens, k = idx.shape
    dx, dw_in, dw_out = np.zeros_like(x), np.zeros_like(w_in), np.zeros_like(w_out)
    dweights = np.zeros((tokens, k))
    for t in range(tokens):
        for j in range(k):
            e = idx[t, j]
            if e < 0:
                continue
            g, u, s = _parts(gu[t, j])
            a = g * s * u
            da = w_out[e].T @ dout[t]
            dweights[t, j] = float(np.dot(da, a))
            da = weights[t, j] * da
            dgu = np.concatenate([da * u * s * (1.0 + g * (1.0 - s)), da * g * s])
            dx[t] += w_in[e].T @ dgu
            dw_in[e] += np.outer(dgu, x[t])
            dw_out[e] += np.outer(dout[t], weights[t, j] * a)
    return dx, dw_in, dw_out, dweights
