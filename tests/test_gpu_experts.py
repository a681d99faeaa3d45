"""The experts' products and their gradient against the float64 oracle.

Tolerances, in norm over a tensor: rounding to bf16 errs by at most 2^-8 of a
value, 2^-8 / sqrt(3) = 2.3e-3 in root mean square over mantissas.  gu, and
f32 weight gradients (one rounded operand): one rounding, 2.5e-3.  out, dx and
bf16 weight gradients: the operand's rounding and the result's, independent,
3.2e-3, held to 3.5e-3.  dweights never leave fp32 products and sums: 1e-5."""
import numpy as np
import pytest
import torch

from newton_schulz_gb300 import binding as B
from oracle import moe_ref as R

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _dev(lib, cuda_ok):
    yield


def _np(t):
    return t.detach().double().cpu().numpy()


def _near(got, want, tol):
    got = _np(got)
    n = np.linalg.norm(want)
    err = np.linalg.norm(got - want)
    assert np.all(np.isfinite(got)) and err <= tol * n, (err, n)


def _data(idx, hidden, inner, experts, seed=1):
    g = torch.Generator().manual_seed(seed)
    tokens, k = idx.shape
    t = lambda *s: torch.randn(*s, generator=g).to(BF16).cuda()  # noqa: E731
    x, dout = t(tokens, hidden), t(tokens, hidden)
    w_in = (torch.randn(experts, 2 * inner, hidden, generator=g) * hidden ** -0.5).to(BF16).cuda()
    w_out = (torch.randn(experts, hidden, inner, generator=g) * inner ** -0.5).to(BF16).cuda()
    idx = idx.to(torch.int32).cuda()
    weights = torch.rand(tokens, k, generator=g).cuda() * (idx >= 0)
    return x, dout, w_in, w_out, B.Route(idx, weights, *B.muon_route_plan(idx, experts))


def _random_idx(tokens, k, experts, seed=0, dropped=0.0):
    g = torch.Generator().manual_seed(seed)
    idx = torch.rand(tokens, experts, generator=g).argsort(1)[:, :k]
    return torch.where(torch.rand(tokens, k, generator=g) < dropped, -1, idx)


def _check(idx, hidden, inner, experts, seed=1, dtypes=(F32, BF16)):
    x, dout, w_in, w_out, r = _data(idx, hidden, inner, experts, seed)
    n = int(r.offsets[-1])
    out, gu = B.muon_experts_forward(x, w_in, w_out, r, save=True)
    i = r.idx.cpu().numpy()
    args = [_np(v) for v in (x, w_in, w_out)]
    want, wgu = R.experts_ref(*args, i, _np(r.weights))
    _near(out, want, 3.5e-3)
    src = r.src.cpu().numpy()[:n]
    rows = wgu.reshape(-1, wgu.shape[2])[src]
    _near(gu[:n], rows, 2.5e-3)
    plain, none = B.muon_experts_forward(x, w_in, w_out, r)
    assert none is None and torch.equal(plain, out)
    saved = np.zeros_like(wgu)
    saved.reshape(-1, wgu.shape[2])[src] = _np(gu[:n])
    grads = R.experts_grad_ref(_np(dout), *args, i, _np(r.weights), saved)
    for dt in dtypes:
        got = B.muon_experts_backward(dout, x, w_in, w_out, r, gu, dw_dtype=dt)
        tol = 2.5e-3 if dt == F32 else 3.5e-3
        for g, w, e in zip(got, grads, (3.5e-3, tol, tol, 1e-5)):
            _near(g, w, e)
        assert bool((got[3][r.pos < 0] == 0).all())
        again = B.muon_experts_backward(dout, x, w_in, w_out, r, gu, dw_dtype=dt)
        assert all(torch.equal(a, b) for a, b in zip(got, again))     # fixed order
    assert B.muon_query_status() == 0


@pytest.mark.parametrize("tokens,k,experts", [(1, 1, 1), (1, 4, 16), (3, 2, 5), (17, 8, 64), (40, 1, 3),
                                              (130, 3, 4), (300, 2, 2)])
@pytest.mark.parametrize("hidden,inner", [(64, 64), (256, 128), (320, 72), (136, 200)])
def test_parity(tokens, k, experts, hidden, inner):
    _check(_random_idx(tokens, k, experts), hidden, inner, experts)


@pytest.mark.parametrize("hidden,inner", [(7, 9), (8, 8), (63, 65), (131, 77), (100, 260), (257, 4)])
def test_odd_widths(hidden, inner):
    _check(_random_idx(50, 2, 4, dropped=0.2), hidden, inner, 4)


@pytest.mark.parametrize("hidden,inner", [(1, 1), (2, 1), (1, 3)])
def test_widths_of_a_few(hidden, inner):
    # a handful of values: no root mean square over mantissas, so the largest
    # error of each rounding, 2^-8 of every term, summed over the terms
    idx = _random_idx(50, 2, 4, dropped=0.2)
    x, dout, w_in, w_out, r = _data(idx, hidden, inner, 4)
    out, gu = B.muon_experts_forward(x, w_in, w_out, r, save=True)
    i, n = r.idx.cpu().numpy(), int(r.offsets[-1])
    args, w = [_np(v) for v in (x, w_in, w_out)], _np(r.weights)
    want, wgu = R.experts_ref(*args, i, w)
    src = r.src.cpu().numpy()[:n]
    saved = np.zeros_like(wgu)
    saved.reshape(-1, 2 * inner)[src] = _np(gu[:n])
    big = [np.abs(a) for a in args]
    def act(g):
        return np.abs(g[..., :inner] / (1 + np.exp(-g[..., :inner])) * g[..., inner:])
    terms = np.zeros_like(want)           # sum of |weight| |W_out| |act|
    for t in range(50):
        for j in range(2):
            if i[t, j] >= 0:
                terms[t] += w[t, j] * (big[2][i[t, j]] @ act(wgu[t, j]))
    assert np.all(np.abs(_np(out) - want) <= 2.0 ** -8 * (terms + np.abs(want)) * 1.01)
    grads = R.experts_grad_ref(_np(dout), *args, i, w, saved)
    got = B.muon_experts_backward(dout, x, w_in, w_out, r, gu)
    t_in, t_out = np.zeros_like(grads[1]), np.zeros_like(grads[2])
    for t in range(50):
        for j in range(2):
            e = i[t, j]
            if e < 0:
                continue
            one = R.experts_grad_ref(_np(dout)[t:t + 1], args[0][t:t + 1], args[1], args[2],
                                     i[t:t + 1, j:j + 1], w[t:t + 1, j:j + 1], saved[t:t + 1, j:j + 1])
            t_in += np.abs(one[1])
            t_out += np.abs(one[2])
    assert np.all(np.abs(_np(got[1]) - grads[1]) <= 2.0 ** -8 * t_in * 1.01)
    assert np.all(np.abs(_np(got[2]) - grads[2]) <= 2.0 ** -8 * t_out * 1.01)


@pytest.mark.parametrize("count", [1, 31, 32, 33, 63, 64, 65, 127, 128, 255, 256, 257, 511, 513, 600])
def test_rows_per_expert_at_tile_borders(count):
    # expert 1 has `count` rows, its neighbours one each, expert 3 none
    idx = torch.cat([torch.zeros(1), torch.ones(count), torch.full((1,), 2.0)]).long()[:, None]
    _check(idx, 72, 40, 4, dtypes=(BF16,))


def test_wide_experts_cross_every_tile():
    _check(_random_idx(70, 2, 3), 600, 520, 3)


def test_many_experts():
    _check(_random_idx(60, 32, 1024), 16, 8, 1024)


def test_dropped_tokens_and_empty_experts():
    idx = _random_idx(64, 4, 16, dropped=0.5)
    idx[:8] = -1
    idx[idx == 5] = -1
    _check(idx, 128, 96, 16)
    x, dout, w_in, w_out, r = _data(idx, 128, 96, 16)
    out, gu = B.muon_experts_forward(x, w_in, w_out, r, save=True)
    dx, dw_in, dw_out, _ = B.muon_experts_backward(dout, x, w_in, w_out, r, gu)
    assert bool((out[:8] == 0).all()) and bool((dx[:8] == 0).all())
    assert bool((dw_in[5] == 0).all()) and bool((dw_out[5] == 0).all())


def test_no_slot_filled_and_no_tokens():
    x, dout, w_in, w_out, r = _data(torch.full((9, 2), -1), 64, 64, 4)
    out, gu = B.muon_experts_forward(x, w_in, w_out, r, save=True)
    got = B.muon_experts_backward(dout, x, w_in, w_out, r, gu)
    assert all(bool((t == 0).all()) for t in (out, *got))
    x, dout, w_in, w_out, r = _data(torch.full((0, 2), -1), 64, 64, 4)
    out, gu = B.muon_experts_forward(x, w_in, w_out, r, save=True)
    got = B.muon_experts_backward(dout, x, w_in, w_out, r, gu)
    assert out.shape == (0, 64) and got[0].shape == (0, 64)
    assert bool((got[1] == 0).all()) and bool((got[2] == 0).all())


def test_strides_and_alignment():
    idx = _random_idx(45, 2, 4)
    x, dout, w_in, w_out, r = _data(idx, 136, 72, 4)
    out, gu = B.muon_experts_forward(x, w_in, w_out, r, save=True)
    want = B.muon_experts_backward(dout, x, w_in, w_out, r, gu)
    def wide(t, off, pad):
        w = torch.full((t.shape[0], off + t.shape[1] + pad), 7.0, dtype=t.dtype, device="cuda")
        w[:, off:off + t.shape[1]] = t
        return w, w[:, off:off + t.shape[1]]
    def odd(t):              # contiguous, but two bytes off a 16-byte boundary
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        b[1:] = t.reshape(-1)
        return b[1:].view(t.shape)
    for off, pad in ((8, 8), (1, 2), (0, 3)):
        _, xv = wide(x, off, pad)
        _, dv = wide(dout, off, pad)
        ow, ov = wide(out * 0, off, pad)
        xw, dxv = wide(out * 0, off, pad)
        B.muon_experts_forward(xv, w_in, w_out, r, out=ov)
        assert torch.equal(ov, out)
        got = B.muon_experts_backward(dv, xv, w_in, w_out, r, gu, dx=dxv)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        for w in (ow, xw):
            assert bool((w[:, :off] == 7).all()) and bool((w[:, off + 136:] == 7).all())
    assert torch.equal(B.muon_experts_forward(x, odd(w_in), odd(w_out), r)[0], out)
    got = B.muon_experts_backward(dout, x, odd(w_in), odd(w_out), r, odd(gu), dw_in=odd(want[1] * 0),
                                  dw_out=odd(want[2] * 0))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_optional_outputs():
    x, dout, w_in, w_out, r = _data(_random_idx(33, 2, 4), 64, 72, 4)
    _, gu = B.muon_experts_forward(x, w_in, w_out, r, save=True)
    full = B.muon_experts_backward(dout, x, w_in, w_out, r, gu)
    a = B.muon_experts_backward(dout, x, w_in, w_out, r, gu, want_dx=False)
    b = B.muon_experts_backward(dout, x, w_in, w_out, r, gu, want_dw=False)
    assert a[0] is None and all(torch.equal(p, q) for p, q in zip(a[1:], full[1:]))
    assert b[1] is None and b[2] is None and torch.equal(b[0], full[0]) and torch.equal(b[3], full[3])


def test_non_finite_tokens_stay_in_their_rows_and_experts():
    idx = torch.arange(40)[:, None] % 4
    x, dout, w_in, w_out, r = _data(idx, 96, 64, 4)
    def run(xx, dd):
        out, gu = B.muon_experts_forward(xx, w_in, w_out, r, save=True)
        return (out, *B.muon_experts_backward(dd, xx, w_in, w_out, r, gu))
    want = run(x, dout)
    bad_x, bad_d = x.clone(), dout.clone()
    bad_x[5, 3], bad_d[9, 1] = float("nan"), float("inf")     # both of expert 1
    got = run(bad_x, bad_d)
    keep = [t for t in range(40) if t not in (5, 9)]
    assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1][keep], want[1][keep])
    for e in (0, 2, 3):
        assert torch.equal(got[2][e], want[2][e]) and torch.equal(got[3][e], want[3][e])
    assert bool(got[0][5].isnan().any())
    # what those calls left in the workspace reaches no later call
    assert all(torch.equal(a, b) for a, b in zip(run(x, dout), want))


def test_wild_plan_entries_are_skipped():
    # a plan that is not one: reads stay inside the tensors
    x, dout, w_in, w_out, r = _data(_random_idx(32, 2, 4), 64, 64, 4)
    out, gu = B.muon_experts_forward(x, w_in, w_out, r, save=True)
    bad = B.Route(r.idx, r.weights, torch.tensor([0, 1 << 30, -5, 7, 1 << 30], dtype=torch.int32).cuda(),
                  torch.full_like(r.src, 1 << 30), torch.full_like(r.pos, 1 << 30))
    o, _ = B.muon_experts_forward(x, w_in, w_out, bad)
    dx, _, _, dwt = B.muon_experts_backward(dout, x, w_in, w_out, bad, gu)
    assert bool((o == 0).all()) and bool((dx == 0).all()) and bool((dwt == 0).all())
    assert torch.equal(B.muon_experts_forward(x, w_in, w_out, r)[0], out)
    assert B.muon_query_status() == 0


def test_side_stream_and_interleaved_sizes():
    big = _data(_random_idx(200, 4, 8), 256, 128, 8)
    small = _data(_random_idx(3, 2, 8, seed=2), 256, 128, 8)
    def run(d, stream=None):
        out, gu = B.muon_experts_forward(d[0], d[2], d[3], d[4], save=True, stream=stream)
        return (out, *B.muon_experts_backward(d[1], d[0], d[2], d[3], d[4], gu, stream=stream))
    want = [run(big), run(small)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [run(small, s), run(big, s), run(small, s)]
    torch.cuda.current_stream().wait_stream(s)
    for g, w in zip(got, (want[1], want[0], want[1])):
        assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_rows_past_32_bit_offsets():
    # 2 * inner * rows = 2.3e9 elements of gu
    tokens, k, hidden, inner, experts = 70_000, 2, 64, 8192, 2
    idx = torch.tensor([[0, 1]]).expand(tokens, k)
    x, _, w_in, w_out, r = _data(idx, hidden, inner, experts)
    out, gu = B.muon_experts_forward(x, w_in, w_out, r, save=True)
    at = [0, 1, 40_000, 65_535, 69_999]
    want, wgu = R.experts_ref(_np(x[at]), _np(w_in), _np(w_out), np.array([[0, 1]] * 5), _np(r.weights[at]))
    _near(out[at], want, 3.5e-3)
    _near(gu[r.pos[at].long()], wgu, 2.5e-3)
