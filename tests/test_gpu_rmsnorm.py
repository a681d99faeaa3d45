"""RMS norm, its 8-bit output and its gradient against the float64 oracle.

Tolerances, from the formats: the fp32 arithmetic of a row (a sum of `cols`
terms in a tree of depth under 30, a root, a division, two products) errs by
under 30 * 2^-24 = 2e-6 of a value (of the row's root mean square where terms
cancel); rounding to bf16 adds at most 2^-8 of the value (nearest even, 8
significant bits); to e4m3 at most 2^-4 of it, or half the spacing 2^-9 of the
subnormal codes.  dgain, a sum over rows, is held in norm: 1e-5."""
import numpy as np
import pytest
import torch

from newton_schulz_gb300 import binding as B
from oracle import moe_ref as R

pytestmark = pytest.mark.gpu
F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
EPS = 1e-6


@pytest.fixture(autouse=True)
def _dev(lib, cuda_ok):
    yield


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def _close(got, want, dtype):
    got, rms = _np(got), np.sqrt((want ** 2).mean(1, keepdims=True)) + 1e-30
    tol = 2e-6 * np.maximum(np.abs(want), rms) + (2.0 ** -8 * np.abs(want) if dtype == BF16 else 0.0)
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)


COLS = [1, 7, 8, 9, 64, 100, 128, 200, 256, 257, 1000, 2048, 4096, 5120, 8192, 16384, 20000, 32768]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("x,res", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, None)])
def test_forward(cols, x, res):
    for rows in (1, 5, 700):      # 700: more rows than the few-rows variant takes
        if rows * cols > 4_000_000 and rows > 5:
            continue
        a, r = _rand((rows, cols), x, 1, 3.0), None if res is None else _rand((rows, cols), res, 2)
        g = _rand((cols,), BF16, 3) if res else None
        y, h, scales = B.muon_rmsnorm_forward(a, g, residual=r, eps=EPS)
        wh, wy = R.rmsnorm_ref(_np(a), _np(r), _np(g), EPS)
        assert scales is None and y.dtype == x
        _close(y, wy, x)
        if res is not None:
            assert h.dtype == res
            _close(h, wh, res)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("cols", [1, 8, 100, 128, 129, 256, 1000, 4096, 8200])
def test_e4m3(cols, group):
    for rows in (3, 900):
        a = _rand((rows, cols), BF16, 4)
        a[0] = 0                                    # an all-zero row
        a[1, cols // 2] = 300.0                     # an outlier
        y, h, s = B.muon_rmsnorm_forward(a, None, eps=EPS, y_dtype=E4M3, group=group)
        assert h is None and s.shape == (rows, -(-cols // group) if group else 1)
        codes, scales = R.e4m3_pieces(R.rmsnorm_ref(_np(a), None, None, EPS)[1], group)
        assert np.all(np.abs(_np(s) - scales) <= 4e-6 * scales)
        got = y.float().cpu().numpy()
        assert np.all(np.abs(got - codes) <= 2.0 ** -4 * np.abs(codes) * (1 + 1e-4) + 2.0 ** -10 + 1e-6)
        assert np.abs(got).max() <= 448 and np.all(got[0] == 0)


@pytest.mark.parametrize("cols", [1, 8, 9, 100, 256, 1000, 4096, 8192, 12000, 20000])
@pytest.mark.parametrize("dt,res", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, None)])
def test_backward(cols, dt, res):
    for rows in (1, 6, 1300):
        if rows * cols > 6_000_000 and rows > 6:
            continue
        dy, h = _rand((rows, cols), dt, 5), _rand((rows, cols), dt, 6, 2.0)
        d = None if res is None else _rand((rows, cols), res, 7)
        g = _rand((cols,), F32, 8)
        dh, dgain = B.muon_rmsnorm_backward(dy, h, g, dres=d, eps=EPS)
        wh, wg = R.rmsnorm_grad_ref(_np(dy), _np(h), _np(g), _np(d), EPS)
        if cols > 1:      # one column: dh is the eps-sized rest of a full cancellation
            rms = np.sqrt((wh ** 2).mean(1, keepdims=True)) + 1e-30
            tol = 4e-6 * np.maximum(np.abs(wh), rms) + (2.0 ** -8 * np.abs(wh) if dt == BF16 else 0)
            assert np.all(np.abs(_np(dh) - wh) <= tol)
        assert np.linalg.norm(_np(dgain) - wg) <= 1e-5 * np.linalg.norm(wg) + 1e-6
        again = B.muon_rmsnorm_backward(dy, h, g, dres=d, eps=EPS)
        assert torch.equal(again[0], dh) and torch.equal(again[1], dgain)     # fixed order


def test_backward_is_the_difference_quotient():
    # f32: f = <dy, y(h)>; a step of 1e-2 errs by about 1e-4 (third derivative)
    # and 2e-6 / 1e-2 (rounding): 2e-3 is held
    h, dy, d = (_rand((64, 512), F32, s) for s in (1, 2, 3))
    g = _rand((512,), F32, 4)
    dh, dgain = B.muon_rmsnorm_backward(dy, h, g, eps=EPS)
    f = lambda v: float((dy.double() * B.muon_rmsnorm_forward(v, g, eps=EPS)[0].double()).sum())  # noqa: E731
    slope = (f(h + 1e-2 * d) - f(h - 1e-2 * d)) / 2e-2
    got = float((dh.double() * d.double()).sum())
    assert abs(got - slope) <= 2e-3 * float(dh.norm()) * float(d.norm()) / 30
    q = lambda v: float((dy.double() * B.muon_rmsnorm_forward(h, v, eps=EPS)[0].double()).sum())  # noqa: E731
    slope = (q(g + 1e-2 * d[0]) - q(g - 1e-2 * d[0])) / 2e-2
    assert abs(float((dgain.double() * d[0].double()).sum()) - slope) <= 2e-3 * abs(slope) + 1e-2


@pytest.mark.parametrize("off,pad", [(0, 8), (1, 3), (4, 0), (3, 5)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_strides_and_alignment(dt, off, pad):
    rows, cols = 37, 264
    def view(seed):
        return _rand((rows, off + cols + pad), dt, seed)[:, off:off + cols]
    x, r, dres = view(1), view(2), view(3)
    g = _rand((cols + 1,), dt, 4)[1:]          # a gain that is not 16-byte aligned
    y = torch.full((rows, off + cols + pad), 7.0, dtype=dt, device="cuda")
    h = torch.full_like(y, 7.0)
    B.muon_rmsnorm_forward(x, g, residual=r, eps=EPS, h=h[:, off:off + cols], y=y[:, off:off + cols])
    wh, wy = R.rmsnorm_ref(_np(x), _np(r), _np(g), EPS)
    _close(y[:, off:off + cols], wy, dt)
    _close(h[:, off:off + cols], wh, dt)
    for t in (y, h):        # nothing outside the view is touched
        assert bool((t[:, :off] == 7).all()) and bool((t[:, off + cols:] == 7).all())
    dh, _ = B.muon_rmsnorm_backward(x, r, g, dres=dres, eps=EPS)
    w, _ = R.rmsnorm_grad_ref(_np(x), _np(r), _np(g), _np(dres), EPS)
    assert np.linalg.norm(_np(dh) - w) <= (4e-3 if dt == BF16 else 4e-6) * np.linalg.norm(w)


def test_in_place_residual_and_gradient():
    x, r, g = _rand((50, 1024), BF16, 1), _rand((50, 1024), BF16, 2), _rand((1024,), BF16, 3)
    y, h, _ = B.muon_rmsnorm_forward(x, g, residual=r, eps=EPS)
    r2 = r.clone()
    y2, h2, _ = B.muon_rmsnorm_forward(x, g, residual=r2, eps=EPS, h=r2)
    assert h2 is r2 and torch.equal(r2, h) and torch.equal(y2, y)
    dh, dg = B.muon_rmsnorm_backward(y, h, g, dres=x, eps=EPS)
    x2 = x.clone()
    dh2, dg2 = B.muon_rmsnorm_backward(y, h, g, dres=x2, eps=EPS, dh=x2)
    assert dh2 is x2 and torch.equal(x2, dh) and torch.equal(dg, dg2)


def test_non_finite_rows_stay_alone():
    x = _rand((20, 300), F32, 1)
    want = B.muon_rmsnorm_forward(x, eps=EPS)[0]
    x[3, 5], x[7, 0] = float("nan"), float("inf")
    y = B.muon_rmsnorm_forward(x, eps=EPS)[0]
    keep = [i for i in range(20) if i not in (3, 7)]
    assert torch.equal(y[keep], want[keep]) and bool(y[3].isnan().all()) and bool(y[7, 0].isnan())


def test_no_rows_and_side_stream():
    e = torch.empty((0, 64), dtype=BF16, device="cuda")
    assert B.muon_rmsnorm_forward(e, eps=EPS)[0].shape == (0, 64)
    dh, dg = B.muon_rmsnorm_backward(e, e, eps=EPS)
    assert dh.shape == (0, 64) and bool((dg == 0).all())
    x, s = _rand((400, 2048), BF16, 1), torch.cuda.Stream()
    want = B.muon_rmsnorm_backward(x, x, eps=EPS)
    s.wait_stream(torch.cuda.current_stream())
    got = B.muon_rmsnorm_backward(x, x, eps=EPS, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_rows_past_32_bit_offsets():
    rows, cols = 140_000, 16_384          # 2.29e9 elements
    x = torch.randn((rows, 1), device="cuda").to(BF16).expand(rows, cols).contiguous()
    x[:, ::2] *= 2
    y = B.muon_rmsnorm_forward(x, eps=EPS)[0]
    at = torch.tensor([0, 1, 131_071, 131_072, 139_999], device="cuda")
    _close(y[at], R.rmsnorm_ref(_np(x[at]), None, None, EPS)[1], BF16)
