"""The block's calls on a stream that is not the current one."""
import pytest
import torch

from newton_schulz_gb300 import binding as B

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _dev(lib, cuda_ok):
    yield


def _randn(*shape, dtype=BF16, seed=1):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def test_outputs_of_a_side_stream_are_its_own():
    # An output allocated for another stream than the call's may be memory that
    # the first still writes: it was freed with a write to it on its way.
    x = _randn(1024, 4096)
    gain = _randn(4096)
    want = B.muon_rmsnorm_forward(x, gain)[0]
    idx = torch.arange(1024, dtype=torch.int32, device="cuda")[:, None] % 4
    cfg = B.make_route_config(512, 8)
    logits = _randn(1024, 512, dtype=F32)
    wr = B.muon_route_forward(logits, cfg)
    route = B.Route(idx, torch.ones(1024, 1, device="cuda"), *B.muon_route_plan(idx, 4))
    w_in, w_out = _randn(4, 128, 4096), _randn(4, 4096, 64)
    wo = B.muon_experts_forward(x, w_in, w_out, route)[0]
    side = torch.cuda.Stream()
    calls = ((lambda: B.muon_rmsnorm_forward(x, gain, stream=side)[0], want),
             (lambda: B.muon_rmsnorm_backward(x, x, gain, stream=side)[0], B.muon_rmsnorm_backward(x, x, gain)[0]),
             (lambda: B.muon_route_forward(logits, cfg, stream=side).weights, wr.weights),
             (lambda: B.muon_experts_forward(x, w_in, w_out, route, stream=side)[0], wo))
    for call, expect in calls:
        torch.cuda.synchronize()
        late = [torch.empty_like(expect) for _ in range(4)]
        torch.cuda._sleep(200_000_000)             # about a tenth of a second
        for t in late:
            t.fill_(7.0)
        del late, t
        got = call()
        torch.cuda.synchronize()
        assert torch.equal(got, expect)


def test_raw_handles_and_positional_streams():
    x = _randn(300, 1000)
    want = B.muon_rmsnorm_forward(x)[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [B.muon_rmsnorm_forward(x, stream=side.cuda_stream)[0], B.muon_rmsnorm_forward(x, stream=0)[0]]
    idx = torch.arange(300, dtype=torch.int32, device="cuda")[:, None] % 7
    torch.cuda.synchronize()
    plans = B.muon_route_plan(idx, 7, side), B.muon_route_plan(idx, 7)
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    assert all(torch.equal(a, b) for a, b in zip(*plans))


def test_current_handle(monkeypatch):
    side = torch.cuda.Stream()
    for drop in (False, True):          # with and without torch's direct way to the handle
        if drop:
            monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
        assert B._current_handle() == torch.cuda.current_stream().cuda_stream
        with torch.cuda.stream(side):
            assert B._current_handle() == side.cuda_stream
