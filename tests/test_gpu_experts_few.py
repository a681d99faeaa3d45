"""The matrix-vector products of a few rows, and which calls take them.  They
keep everything in fp32 up to the result: out is the exact sum rounded to bf16
once.  So its distance from 64 bits is that of the rounded exact values; the fp32
sums (2048 and 768 terms in trees, random signs) err by a few 2^-24 sqrt(terms),
under 1e-5 in norm, and turn a few roundings over: 2 % and 2e-5 are allowed
beside it."""
import pytest
import torch

from newton_schulz_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _dev(lib, cuda_ok):
    yield


@pytest.mark.parametrize("tokens,k,experts", [(1, 8, 20), (1, 1, 1), (4, 2, 8), (8, 2, 32), (1, 32, 40)])
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


# (tokens, top_k, experts): launches.  An expert of [768, 2048] is 9.4 MB, of
# [64, 256] 0.1 MB; rows beyond the experts they hit read that much again.
@pytest.mark.parametrize("tokens,k,experts,hidden,inner,launches", [
    (1, 8, 64, 2048, 768, 2), (4, 2, 8, 2048, 768, 2), (8, 2, 8, 2048, 768, 4), (16, 2, 8, 2048, 768, 4),
    (16, 2, 8, 256, 64, 2), (17, 2, 8, 256, 64, 4), (32, 1, 1, 256, 64, 2), (32, 1, 1, 2048, 768, 4)])
def test_rows_that_share_wide_experts_go_by_tiles(tokens, k, experts, hidden, inner, launches):
    g = torch.Generator("cuda").manual_seed(1)
    t = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale).to(BF16)  # noqa: E731
    x, w_in = t(tokens, hidden), t(experts, 2 * inner, hidden, scale=hidden ** -0.5)
    w_out = t(experts, hidden, inner, scale=inner ** -0.5)
    idx = torch.rand(tokens, experts, generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32)
    r = B.Route(idx, torch.ones(tokens, k, device="cuda"), *B.muon_route_plan(idx, experts))
    out = B.muon_experts_forward(x, w_in, w_out, r)[0].double()
    assert B.muon_last_launch_count() == launches
    want = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda")
    for i in range(tokens):
        for e in idx[i].tolist():
            v = w_in[e].double() @ x[i].double()
            want[i] += w_out[e].double() @ (v[:inner] * torch.sigmoid(v[:inner]) * v[inner:])
    assert float((out - want).norm()) <= 3.5e-3 * float(want.norm())      # as test_gpu_experts derives
