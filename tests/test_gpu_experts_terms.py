"""The slot products' storage between the experts' products and the sum over
slots (dx's terms likewise): features far larger than their neighbours, and
values that are not finite.

Tolerances, per feature (a column of out or dx): the rounding of the product's
operand to bf16 and of the result, each at most 2^-8 / sqrt(3) in root mean
square over mantissas, independent: 3.2e-3, held to 3.5e-3 as for a whole
tensor; a term's own rounding is to be small beside them whatever the other
features hold."""
import pytest
import torch

from newton_schulz_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _dev(lib, cuda_ok):
    yield


def _case(tokens, k, hidden, inner, experts, seed=1):
    g = torch.Generator().manual_seed(seed)
    t = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(BF16).cuda()  # noqa: E731
    x, dout = t(tokens, hidden), t(tokens, hidden)
    w_in = t(experts, 2 * inner, hidden, scale=hidden ** -0.5)
    w_out = t(experts, hidden, inner, scale=inner ** -0.5)
    idx = torch.rand(tokens, experts, generator=g).argsort(1)[:, :k].to(torch.int32).cuda()
    weights = torch.rand(tokens, k, generator=g).cuda() + 0.1
    return x, dout, w_in, w_out, B.Route(idx, weights, *B.muon_route_plan(idx, experts))


def _formulas(x, w_in, w_out, r, dout, gu):
    """out, and dx from the saved gu, in 64 bits."""
    inner = w_out.shape[2]
    out, dx = torch.zeros_like(x, dtype=torch.float64), torch.zeros_like(x, dtype=torch.float64)
    for e in range(w_in.shape[0]):
        t, j = (r.idx == e).nonzero(as_tuple=True)
        w = r.weights[t, j].double()[:, None]
        v = x[t].double() @ w_in[e].double().T
        act = v[:, :inner] * torch.sigmoid(v[:, :inner]) * v[:, inner:]
        out.index_add_(0, t, w * (act @ w_out[e].double().T))
        g, u = gu[r.pos[t, j].long()].double().split(inner, 1)
        s = torch.sigmoid(g)
        da = w * (dout[t].double() @ w_out[e].double())
        dx.index_add_(0, t, torch.cat([da * u * s * (1 + g * (1 - s)), da * g * s], 1) @ w_in[e].double())
    return out, dx


@pytest.mark.parametrize("ratio", [1024.0, 2.0 ** 20])
@pytest.mark.parametrize("hidden,inner", [(256, 128), (200, 72)])
def test_large_features_leave_their_neighbours_alone(ratio, hidden, inner):
    x, dout, w_in, w_out, r = _case(300, 3, hidden, inner, 4)
    # powers of two, so nothing else changes: feature h of out and of dx grow
    big = torch.arange(5, hidden, 32, device="cuda")
    w_out[:, big] *= ratio
    dout[:, big] /= ratio
    w_in[:, :, big] *= ratio
    x[:, big] /= ratio
    out, gu = B.muon_experts_forward(x, w_in, w_out, r, save=True)
    dx = B.muon_experts_backward(dout, x, w_in, w_out, r, gu, want_dw=False)[0]
    for got, want in zip((out, dx), _formulas(x, w_in, w_out, r, dout, gu)):
        err, size = (got.double() - want).norm(dim=0), want.norm(dim=0)
        assert bool((err <= 3.5e-3 * size).all()), float((err / size).max())
    assert B.muon_query_status() == 0


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("tokens", [16, 17, 300])      # 32 rows go to the matrix-vector kernels
def test_a_non_finite_feature_stays_alone(value, tokens):
    x, dout, w_in, w_out, r = _case(tokens, 2, 96, 64, 4)
    hit = (r.idx == 1).any(1)
    out, gu = B.muon_experts_forward(x, w_in, w_out, r, save=True)
    dx = B.muon_experts_backward(dout, x, w_in, w_out, r, gu, want_dw=False)[0]
    bad_out, bad_in = w_out.clone(), w_in.clone()
    bad_out[1, 37, 8] = value          # feature 37 of out, through expert 1
    bad_in[1, 5, 70] = value           # feature 70 of dx, likewise
    got = (B.muon_experts_forward(x, w_in, bad_out, r)[0],
           B.muon_experts_backward(dout, x, bad_in, w_out, r, gu, want_dw=False)[0])
    for a, want, col in zip(got, (out, dx), (37, 70)):
        rest = [c for c in range(96) if c != col]
        assert torch.equal(a[:, rest], want[:, rest])
        assert torch.equal(a[~hit, col], want[~hit, col])
        one = a[hit, col]
        assert bool((one.isnan() if value != value else one.isinf()).all())
