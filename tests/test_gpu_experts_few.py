"""The matrix-vector products of at most 32 rows keep everything in fp32 up to
the result: out is the exact sum rounded to bf16 once.  So its distance from 64
bits is that of the rounded exact values; the fp32 sums (2048 and 768 terms in
trees, random signs) err by a few 2^-24 sqrt(terms), under 1e-5 in norm, and
turn a few roundings over: 2 % and 2e-5 are allowed beside it."""
import pytest
import torch

from newton_schulz_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _dev(lib, cuda_ok):
    yield


@pytest.mark.parametrize("tokens,k,experts", [(1, 8, 20), (1, 1, 1), (4, 2, 8), (16, 2, 8), (1, 32, 40)])
@pytest.mark.parametrize("hidden,inner", [(2048, 768), (1000, 1160), (131, 77), (64, 20)])
def test_one_rounding(tokens, k, experts, hidden, inner):
    g = torch.Generator().manual_seed(tokens + hidden)
    t = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(BF16).cuda()  # noqa: E731
    x = t(tokens, hidden)
    w_in = t(experts, 2 * inner, hidden, scale=hidden ** -0.5)
    w_out = t(experts, hidden, inner, scale=inner ** -0.5)
    idx = torch.rand(tokens, experts, generator=g).argsort(1)[:, :k].to(torch.int32).cuda()
    weights = torch.rand(tokens, k, generator=g).cuda()
    r = B.Route(idx, weights, *B.muon_route_plan(idx, experts))
    out = B.muon_experts_forward(x, w_in, w_out, r)[0].double()
    want = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda")
    for i in range(tokens):
        for j in range(k):
            e = int(idx[i, j])
            v = w_in[e].double() @ x[i].double()
            act = v[:inner] * torch.sigmoid(v[:inner]) * v[inner:]
            want[i] += weights[i, j].double() * (w_out[e].double() @ act)
    rounding = float((want.to(BF16).double() - want).norm())
    assert float((out - want).norm()) <= 1.02 * rounding + 2e-5 * float(want.norm())
