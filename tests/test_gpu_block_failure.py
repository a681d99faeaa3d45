"""The failure path of the bounded waits in the mixture-of-experts block's
kernels, by the library's testing hook (test_gpu_failure has the optimizer's):
the call returns, the status word reports the timeout once, and the next clean
call gives the bits of one made before.  The bound is 50 ms for the stalled
launch."""
import pytest
import torch

from newton_schulz_gb300 import binding as B

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TIMEOUT = 6


@pytest.fixture(autouse=True)
def _dev(lib, cuda_ok):
    yield
    B.muon_debug_inject_stall(B.INJECT_NONE)
    torch.cuda.synchronize()
    assert B.muon_query_status() in (0, TIMEOUT)


def _randn(*shape, dtype=BF16, seed=1):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def _stall(call, monkeypatch):
    want = call()
    torch.cuda.synchronize()
    assert B.muon_query_status() == 0
    monkeypatch.setenv("MUON_WAIT_TIMEOUT_MS", "50")
    B.muon_debug_inject_stall(B.INJECT_GEMM)
    call()
    torch.cuda.synchronize()
    assert B.muon_query_status() == TIMEOUT
    assert B.muon_query_status() == 0
    monkeypatch.delenv("MUON_WAIT_TIMEOUT_MS")
    again = call()
    torch.cuda.synchronize()
    assert B.muon_query_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, again))


@pytest.mark.parametrize("cols,dtype", [(4096, BF16), (8192, BF16), (1000, F32)])
def test_norm_gradient_ring(cols, dtype, monkeypatch):
    dy, h, gain = _randn(3000, cols, dtype=dtype), _randn(3000, cols, dtype=dtype, seed=2), _randn(cols, seed=3)
    _stall(lambda: B.muon_rmsnorm_backward(dy, h, gain, dres=dy), monkeypatch)


# hidden and inner that take one pair, and clusters of two
@pytest.mark.parametrize("tokens,hidden,inner", [(300, 256, 136), (1500, 1024, 1024)])
@pytest.mark.parametrize("back", [False, True])
def test_experts_products(tokens, hidden, inner, back, monkeypatch):
    idx = torch.stack([torch.arange(tokens) % 3, torch.full((tokens,), 4)], 1).to(torch.int32).cuda()
    r = B.Route(idx, _randn(tokens, 2, dtype=F32).abs(), *B.muon_route_plan(idx, 5))      # expert 3 has no rows
    x, dout = _randn(tokens, hidden), _randn(tokens, hidden, seed=2)
    w_in = _randn(5, 2 * inner, hidden, seed=3) * hidden ** -0.5
    w_out = _randn(5, hidden, inner, seed=4) * inner ** -0.5
    if not back:
        _stall(lambda: B.muon_experts_forward(x, w_in, w_out, r)[:1], monkeypatch)
        return
    gu = B.muon_experts_forward(x, w_in, w_out, r, save=True)[1]
    _stall(lambda: B.muon_experts_backward(dout, x, w_in, w_out, r, gu), monkeypatch)
