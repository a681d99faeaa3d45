"""RMS norm in the launch forms that the sizes of test_gpu_rmsnorm do not reach:
the gradient's ring with four chunks a thread (rows of 4104 to 8192 columns),
its register form with several rows a slot (wide, odd or unaligned rows of
large batches), in place and strided through the ring, and rows of several
chunks forward.  Against the formulas in 64 bits on the device; tolerances as
derived in test_gpu_rmsnorm."""
import pytest
import torch

from newton_schulz_gb300 import binding as B

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-6


@pytest.fixture(autouse=True)
def _dev(lib, cuda_ok):
    yield


def _rand(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda") * scale).to(dtype)


def _gradient(dy, h, gain, dres):
    dy, h, gain = dy.double(), h.double(), gain.double()
    inv = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    u, g = h * inv, dy * gain
    dh = inv * (g - u * (g * u).mean(1, keepdim=True))
    return dh if dres is None else dh + dres.double(), (dy * u).sum(0)


def _hold(dh, dgain, want, wgain):
    rms = (want * want).mean(1, keepdim=True).sqrt() + 1e-30
    tol = 4e-6 * torch.maximum(want.abs(), rms)
    if dh.dtype == BF16:
        tol = tol + 2.0 ** -8 * want.abs()
    assert bool(((dh.double() - want).abs() <= tol).all())
    assert float((dgain.double() - wgain).norm()) <= 1e-5 * float(wgain.norm())


@pytest.mark.parametrize("rows,cols,dy,h,res", [
    (1300, 8192, BF16, BF16, BF16), (1300, 8192, BF16, BF16, None), (1300, 4104, BF16, BF16, F32),
    (1300, 4104, BF16, F32, None), (2500, 5120, BF16, BF16, BF16), (1300, 8192, F32, F32, F32),
    (1300, 12000, BF16, BF16, BF16), (1300, 12000, F32, F32, F32), (3000, 4097, BF16, BF16, F32),
    (3000, 4097, F32, F32, None), (5000, 1000, F32, F32, F32), (5000, 1001, BF16, BF16, BF16),
    (20000, 72, BF16, BF16, BF16), (20000, 9, F32, BF16, None), (1300, 32768, BF16, BF16, BF16),
    (1217, 2048, BF16, BF16, BF16), (1216, 528, F32, BF16, BF16)])
def test_gradient(rows, cols, dy, h, res):
    a, b, g = _rand((rows, cols), dy, 1), _rand((rows, cols), h, 2, 2.0), _rand((cols,), F32, 3)
    d = None if res is None else _rand((rows, cols), res, 4)
    got = B.muon_rmsnorm_backward(a, b, g, dres=d, eps=EPS)
    _hold(*got, *_gradient(a, b, g, d))
    again = B.muon_rmsnorm_backward(a, b, g, dres=d, eps=EPS)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    assert B.muon_query_status() == 0


@pytest.mark.parametrize("cols", [4096, 8192])
@pytest.mark.parametrize("off,pad", [(0, 8), (8, 16), (1, 0)])
def test_gradient_of_views(cols, off, pad):
    def view(seed):
        return _rand((2000, off + cols + pad), BF16, seed)[:, off:off + cols]
    dy, h, d = view(1), view(2), view(3)
    g = _rand((cols,), BF16, 4)
    out = torch.full((2000, off + cols + pad), 7.0, dtype=BF16, device="cuda")
    dh, dgain = B.muon_rmsnorm_backward(dy, h, g, dres=d, eps=EPS, dh=out[:, off:off + cols])
    _hold(dh, dgain, *_gradient(dy, h, g, d))
    assert bool((out[:, :off] == 7).all()) and bool((out[:, off + cols:] == 7).all())


@pytest.mark.parametrize("cols", [2048, 4096, 8192, 12000])
def test_gradient_in_place(cols):
    dy, h, d = (_rand((2600, cols), BF16, s) for s in (1, 2, 3))
    g = _rand((cols,), BF16, 4)
    want = B.muon_rmsnorm_backward(dy, h, g, dres=d, eps=EPS)
    dres = d.clone()
    got = B.muon_rmsnorm_backward(dy, h, g, dres=dres, eps=EPS, dh=dres)
    assert torch.equal(dres, want[0]) and torch.equal(got[1], want[1])
    over = dy.clone()
    got = B.muon_rmsnorm_backward(over, h, g, dres=d, eps=EPS, dh=over)
    assert torch.equal(over, want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("rows,cols,x,res", [
    (1300, 8192, BF16, BF16), (1300, 8192, F32, F32), (1300, 12000, BF16, F32), (3000, 4097, BF16, BF16),
    (1300, 32768, F32, F32), (5000, 1001, F32, None), (20000, 72, BF16, BF16), (20000, 9, BF16, None)])
def test_forward(rows, cols, x, res):
    a, g = _rand((rows, cols), x, 1, 3.0), _rand((cols,), F32, 3)
    r = None if res is None else _rand((rows, cols), res, 2)
    y, h, _ = B.muon_rmsnorm_forward(a, g, residual=r, eps=EPS)
    wh = a.double() if r is None else a.double() + r.double()
    wy = wh * torch.rsqrt((wh * wh).mean(1, keepdim=True) + EPS) * g.double()
    for got, want in ((y, wy), (h, wh)):
        if got is None:
            continue
        rms = (want * want).mean(1, keepdim=True).sqrt() + 1e-30
        tol = 2e-6 * torch.maximum(want.abs(), rms)
        if got.dtype == BF16:
            tol = tol + 2.0 ** -8 * want.abs()
        assert bool(((got.double() - want).abs() <= tol).all())
