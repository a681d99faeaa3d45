"""Outputs that share a buffer with inputs without sharing an element (column
ranges of one matrix)."""
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


def test_columns_of_one_buffer_do_not_overlap():
    buf = _randn(50, 400)
    x, y = buf[:, :200], buf[:, 200:]
    want = B.muon_rmsnorm_forward(x.clone())[0]
    B.muon_rmsnorm_forward(x, y=y)
    assert torch.equal(y, want)
    dh = B.muon_rmsnorm_backward(x.clone(), want)[0]
    wide = _randn(50, 600)
    wide[:, 100:300] = x
    B.muon_rmsnorm_backward(wide[:, 100:300], want, dh=wide[:, 300:500])
    assert torch.equal(wide[:, 300:500], dh)
    cfg = B.make_route_config(40, 4)
    logits = _randn(50, 100, dtype=F32)
    r = B.muon_route_forward(logits[:, :40], cfg)
    dw = _randn(50, 4, dtype=F32, seed=2)
    grad = B.muon_route_backward(logits[:, :40].clone(), cfg, r.idx, dw)
    B.muon_route_backward(logits[:, :40], cfg, r.idx, dw, dlogits=logits[:, 50:90])
    assert torch.equal(logits[:, 50:90], grad)
    idx = torch.arange(50, dtype=torch.int32, device="cuda")[:, None] % 4
    route = B.Route(idx, _randn(50, 1, dtype=F32).abs(), *B.muon_route_plan(idx, 4))
    w_in, w_out = _randn(4, 96, 64), _randn(4, 64, 48)
    both = _randn(50, 128)
    out = B.muon_experts_forward(both[:, :64].clone(), w_in, w_out, route)[0]
    B.muon_experts_forward(both[:, :64], w_in, w_out, route, out=both[:, 64:])
    assert torch.equal(both[:, 64:], out)


def test_columns_that_share_elements_are_refused():
    buf = _randn(50, 400)
    for a, b in ((slice(0, 200), slice(199, 399)), (slice(10, 210), slice(0, 200)), (slice(0, 200), slice(0, 200)),
                 (slice(100, 300), slice(0, 200))):
        with pytest.raises(B.MuonError, match="ALIAS"):
            B.muon_rmsnorm_forward(buf[:, a], y=buf[:, b])
    rows = _randn(60, 200)
    with pytest.raises(B.MuonError, match="ALIAS"):       # ten rows on
        B.muon_rmsnorm_forward(rows[:50], y=rows[10:])
    with pytest.raises(B.MuonError, match="ALIAS"):       # a row's end is the next one's start
        B.muon_rmsnorm_forward(buf.view(-1)[:400 * 49].view(49, 400)[:, :300],
                               y=buf.view(-1)[200:200 + 400 * 49].view(49, 400)[:, :300])
    with pytest.raises(B.MuonError, match="ALIAS"):       # another stride
        B.muon_rmsnorm_forward(buf[:, :100], y=buf.view(-1)[100:100 + 50 * 300].view(50, 300)[:, :100])
