"""Workspace guard bands (test_gpu_guard has what they are) behind every buffer
that the mixture-of-experts block's calls lay out: each call leaves its bands
intact, is checked (the check's kernel runs), and gives the same bits."""
import pytest
import torch
from torch.profiler import ProfilerActivity, profile

from newton_schulz_gb300 import binding as B

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _dev(lib, cuda_ok):
    yield
    torch.cuda.synchronize()


def _randn(*shape, dtype=BF16, seed=1):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def _norm(rows, cols):
    dy, h, gain = _randn(rows, cols), _randn(rows, cols, seed=2), _randn(cols, seed=3)
    return lambda: B.muon_rmsnorm_backward(dy, h, gain)


def _route(plan_only):
    logits, cfg = _randn(1000, 96, dtype=F32), B.make_route_config(96, 6)
    r = B.muon_route_forward(logits, cfg)
    return (lambda: B.muon_route_plan(r.idx, 96)) if plan_only else (lambda: B.muon_route_forward(logits, cfg))


def _experts(tokens, hidden, inner, experts, back):
    idx = torch.rand(tokens, experts, generator=torch.Generator().manual_seed(1)).argsort(1)[:, :2]
    idx = torch.where(torch.rand(tokens, 2, generator=torch.Generator().manual_seed(2)) < 0.1, -1, idx)
    idx = idx.to(torch.int32).cuda()
    r = B.Route(idx, _randn(tokens, 2, dtype=F32).abs(), *B.muon_route_plan(idx, experts))
    x, dout = _randn(tokens, hidden), _randn(tokens, hidden, seed=2)
    w_in, w_out = _randn(experts, 2 * inner, hidden, seed=3), _randn(experts, hidden, inner, seed=4)
    n = int(r.offsets[-1])      # later rows of gu are not written
    if not back:
        def run():
            out, gu = B.muon_experts_forward(x, w_in, w_out, r, save=True)
            return out, gu[:n]
        return run
    gu = B.muon_experts_forward(x, w_in, w_out, r, save=True)[1]
    return lambda: B.muon_experts_backward(dout, x, w_in, w_out, r, gu)


CASES = {
    "norm gradient": (_norm, 300, 1000), "norm gradient ring": (_norm, 2000, 2048),
    "route": (_route, False), "plan": (_route, True),
    "few": (_experts, 7, 200, 77, 5, False), "tiles": (_experts, 300, 264, 136, 5, False),
    "odd": (_experts, 90, 131, 77, 5, False), "clusters": (_experts, 900, 1024, 1032, 3, False),
    "gradient": (_experts, 300, 264, 136, 5, True), "odd gradient": (_experts, 90, 131, 77, 5, True),
    "few gradient": (_experts, 3, 64, 64, 40, True), "copy beside": (_experts, 8300, 136, 72, 9, True),
}


@pytest.fixture(scope="module")
def profiler(cuda_ok):
    """A process's first profile may record nothing."""
    with profile(activities=[ProfilerActivity.CUDA]):
        torch.zeros(1, device="cuda")
        torch.cuda.synchronize()


@pytest.mark.parametrize("name", CASES)
def test_bands_intact_and_results_unchanged(name, profiler, monkeypatch):
    call = CASES[name][0](*CASES[name][1:])
    want = call()
    B.muon_release_workspace()
    monkeypatch.setenv("MUON_WS_GUARD", "1")
    with profile(activities=[ProfilerActivity.CUDA]) as prof:
        got = call()
        torch.cuda.synchronize()
    kernels = [e.name for e in prof.events()]
    assert not kernels or any("guard_check" in k for k in kernels)
    assert B.muon_query_status() == 0
    assert B.muon_debug_guard_check() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))
