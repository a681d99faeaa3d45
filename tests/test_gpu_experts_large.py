"""The experts' products where their launches take another form: clusters of
two CTA pairs (256 rows an expert and 1024 of K or more), a row copy beside
the gradient's product (16384 rows or more), and the border between the
matrix-vector products of a few rows and the tiles.  Against the formulas in
64 bits, an expert at a time.

Tolerances as derived in test_gpu_experts: gu and f32 weight gradients 2.5e-3
(one rounding to bf16), out, dx and bf16 weight gradients 3.5e-3 (two),
dweights 1e-5, all in norm over a tensor."""
import pytest
import torch

from newton_schulz_gb300 import binding as B

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _dev(lib, cuda_ok):
    yield


def _near(got, want, tol):
    got = got.double()
    assert bool(torch.isfinite(got).all())
    err, n = float((got - want).norm()), float(want.norm())
    assert err <= tol * n, (err, n)


def _formulas(x, dout, w_in, w_out, idx, weights, saved):
    """out, gu and the gradients in 64 bits; the gradients from the saved gu [tokens, k, 2 inner]."""
    x, dout, weights = x.double(), dout.double(), weights.double()
    tokens, k = idx.shape
    inner = w_out.shape[2]
    out, dx, dwt = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(weights)
    gu = torch.zeros(tokens, k, 2 * inner, dtype=torch.float64, device=x.device)
    dw_in = torch.zeros(w_in.shape, dtype=torch.float64, device=x.device)
    dw_out = torch.zeros(w_out.shape, dtype=torch.float64, device=x.device)
    for e in range(w_in.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        wi, wo, w = w_in[e].double(), w_out[e].double(), weights[t, j][:, None]
        v = x[t] @ wi.T
        gu[t, j] = v
        out.index_add_(0, t, w * ((v[:, :inner] * torch.sigmoid(v[:, :inner]) * v[:, inner:]) @ wo.T))
        g, u = saved[t, j].double().split(inner, 1)
        s = torch.sigmoid(g)
        a, da = g * s * u, dout[t] @ wo
        dwt[t, j] = (da * a).sum(1)
        dgu = w * torch.cat([da * u * s * (1 + g * (1 - s)), da * g * s], 1)
        dx.index_add_(0, t, dgu @ wi)
        dw_in[e] = dgu.T @ x[t]
        dw_out[e] = dout[t].T @ (w * a)
    return out, gu, dx, dw_in, dw_out, dwt


def _check(idx, hidden, inner, experts, dtypes=(F32, BF16)):
    g = torch.Generator().manual_seed(3)
    tokens, k = idx.shape
    t = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(BF16).cuda()  # noqa: E731
    x, dout = t(tokens, hidden), t(tokens, hidden)
    w_in = t(experts, 2 * inner, hidden, scale=hidden ** -0.5)
    w_out = t(experts, hidden, inner, scale=inner ** -0.5)
    idx = idx.to(torch.int32).cuda()
    weights = torch.rand(tokens, k, generator=g).cuda() * (idx >= 0)
    r = B.Route(idx, weights, *B.muon_route_plan(idx, experts))
    out, gu = B.muon_experts_forward(x, w_in, w_out, r, save=True)
    saved = gu[r.pos.clamp(min=0).long()]
    want = _formulas(x, dout, w_in, w_out, idx, weights, saved)
    _near(out, want[0], 3.5e-3)
    _near(torch.where(r.pos[:, :, None] >= 0, saved, 0), want[1], 2.5e-3)
    assert torch.equal(B.muon_experts_forward(x, w_in, w_out, r)[0], out)
    for dt in dtypes:
        got = B.muon_experts_backward(dout, x, w_in, w_out, r, gu, dw_dtype=dt)
        tol = 2.5e-3 if dt == F32 else 3.5e-3
        for a, b, e in zip(got, want[2:], (3.5e-3, tol, tol, 1e-5)):
            _near(a, b, e)
        again = B.muon_experts_backward(dout, x, w_in, w_out, r, gu, dw_dtype=dt)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert B.muon_query_status() == 0


def _counts(*rows):
    return torch.cat([torch.full((n,), e) for e, n in enumerate(rows)]).long()[:, None]


# 1400 and 2320 columns: six and ten M tiles; 2100 and 2208: nine, so that the
# last cluster's second pair has no columns
@pytest.mark.parametrize("hidden,inner", [(1400, 1160), (2100, 1100)])
@pytest.mark.parametrize("rows", [(1100, 1030), (2033, 0, 20, 3000, 65)])
def test_clusters_of_two_pairs(hidden, inner, rows):
    _check(_counts(*rows), hidden, inner, len(rows))


def test_clusters_with_odd_widths():
    _check(_counts(700, 513), 1537, 1283, 2, dtypes=(BF16,))


@pytest.mark.parametrize("experts", [8, 9, 40])
@pytest.mark.parametrize("hidden,inner", [(72, 40), (264, 136)])
def test_copies_beside_products(experts, hidden, inner):
    g = torch.Generator().manual_seed(experts)
    idx = torch.rand(8200, experts, generator=g).argsort(1)[:, :2]
    _check(torch.where(torch.rand(8200, 2, generator=g) < 0.0005, -1, idx), hidden, inner, experts, dtypes=(BF16,))


@pytest.mark.parametrize("rows", [(0,) * 8 + (16400,), (16400,) + (0,) * 8, (1, 16384, 0, 0, 0, 0, 0, 0, 31)])
def test_copies_beside_products_of_lopsided_routings(rows):
    _check(_counts(*rows), 96, 64, 9, dtypes=(BF16,))


@pytest.mark.parametrize("tokens", [1, 2, 15, 16, 17, 18])
@pytest.mark.parametrize("hidden,inner", [(2048, 72), (200, 1100), (133, 70)])
def test_border_of_a_few_rows(tokens, hidden, inner):
    g = torch.Generator().manual_seed(tokens)
    _check(torch.rand(tokens, 6, generator=g).argsort(1)[:, :2], hidden, inner, 6, dtypes=(BF16,))
