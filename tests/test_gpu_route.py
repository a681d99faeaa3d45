"""Routing, its row plan and its gradient against the float64 oracle.

The choice and the plan are whole numbers and must be equal: logits come from
a grid of spacing 1/64 without repeats in a row (or with deliberate repeats),
biases from a grid of 2^-10 on sigmoid scores, so that no two keys are within
rounding of each other unless they are equal.  Weights: an exponential, a sum
of at most 1024 terms and two divisions in fp32, under 2e-6 of a weight; the
gradient's differences are held to 4e-6 of the row's largest value (bf16: 2^-8
of the value more)."""
import numpy as np
import pytest
import torch

from newton_schulz_gb300 import binding as B
from oracle import moe_ref as R

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
NAMES = {"softmax": B.ROUTE_SOFTMAX, "sigmoid": B.ROUTE_SIGMOID, "max": B.GROUP_MAX, "sum2": B.GROUP_SUM2}


@pytest.fixture(autouse=True)
def _dev(lib, cuda_ok):
    yield


def _np(t):
    return t.detach().double().cpu().numpy()


def _logits(tokens, experts, seed, dtype=F32):
    """Distinct values per row, multiples of 1/64 (exact in bf16 within +-4 for up to 512 experts)."""
    r = np.random.default_rng(seed)
    grid = (np.arange(experts) - experts // 2) / 64.0
    rows = np.stack([r.permutation(grid) for _ in range(tokens)])
    return torch.tensor(rows, dtype=dtype).cuda()


def _check(logits, k, bias=None, mask=None, **cfg):
    c = B.make_route_config(logits.shape[1], k, score=NAMES[cfg.get("score", "softmax")],
                            groups=cfg.get("groups", 1), top_groups=cfg.get("top_groups"),
                            group_score=NAMES[cfg.get("group_score", "max")],
                            renormalize=cfg.get("renormalize", False), scale=cfg.get("scale", 1.0))
    r = B.muon_route_forward(logits, c, bias=bias, mask=mask)
    idx, w = R.route_ref(_np(logits), k, bias=None if bias is None else _np(bias),
                         mask=None if mask is None else mask.cpu().numpy(), **cfg)
    assert np.array_equal(r.idx.cpu().numpy(), idx)
    assert np.all(np.abs(_np(r.weights) - w) <= 2e-6 * np.abs(w) + 1e-30)
    for got, want in zip((r.offsets, r.src, r.pos), R.plan_ref(idx, logits.shape[1])):
        assert np.array_equal(got.cpu().numpy(), want)
    return r, c


@pytest.mark.parametrize("experts", [1, 2, 5, 31, 32, 33, 64, 100, 128, 160, 256, 257, 512, 1000, 1024])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choice_weights_plan(experts, score):
    for tokens, k in ((1, 1), (9, min(8, experts)), (40, min(32, experts))):
        _check(_logits(tokens, experts, tokens + experts), k, score=score,
               renormalize=tokens == 9, scale=2.5 if tokens == 9 else 1.0)


@pytest.mark.parametrize("tokens", [255, 256, 257, 700, 1025])
def test_many_tokens(tokens):
    mask = torch.rand(tokens, generator=torch.Generator().manual_seed(1)).cuda() < 0.8
    _check(_logits(tokens, 40, 3, BF16), 5, mask=mask, score="sigmoid", renormalize=True)


@pytest.mark.parametrize("groups,top", [(2, 1), (8, 4), (8, 1), (64, 3), (4, 4)])
@pytest.mark.parametrize("rank", ["max", "sum2"])
@pytest.mark.parametrize("biased", [False, True])
def test_groups_and_bias(groups, top, rank, biased):
    r = np.random.default_rng(5)
    # a bias of odd multiples of 2^-11: no sum of scores and biases repeats
    bias = torch.tensor((2 * r.permutation(128) - 127) / 2048.0, dtype=F32).cuda() if biased else None
    k = min(6, 128 // groups * top)
    _check(_logits(33, 128, 6), k, bias=bias, score="sigmoid", groups=groups, top_groups=top,
           group_score=rank, renormalize=True)


def test_ties_go_to_the_lowest_index():
    r = np.random.default_rng(7)
    x = torch.tensor(r.integers(-2, 3, (64, 96)) / 2.0, dtype=BF16).cuda()
    for cfg in (dict(), dict(groups=8, top_groups=2), dict(groups=8, top_groups=3, score="sigmoid")):
        _check(x, 8, **cfg)
    _check(torch.zeros(3, 70).cuda(), 9)
    # -0 and +0 are equal
    z = torch.zeros(2, 40)
    z[:, ::2] = -0.0
    _check(z.cuda(), 5)


def test_masked_experts_and_tokens():
    inf = float("inf")
    x = _logits(12, 64, 8)
    x[0] = -inf                                   # nothing left
    x[1, 3:] = -inf                               # fewer experts than slots
    x[2, :] = torch.finfo(F32).min                # the type's lowest value is a value
    x[3, ::2] = torch.finfo(F32).min
    x[4, 32:] = -inf                              # half the groups empty
    mask = torch.ones(12, dtype=torch.bool, device="cuda")
    mask[5] = False
    for cfg in (dict(), dict(score="sigmoid", renormalize=True), dict(groups=4, top_groups=2),
                dict(groups=4, top_groups=3, group_score="sum2", score="sigmoid")):
        r, _ = _check(x, 6, mask=mask, **cfg)
        assert bool((r.idx[0] == -1).all()) and bool((r.idx[5] == -1).all())
    _check(x, 6, mask=torch.zeros(12, dtype=torch.uint8, device="cuda"))     # every token left out
    assert B.muon_query_status() == 0


def test_non_finite_logits_set_the_status():
    x = _logits(4, 48, 9)
    x[1, 7], x[2, 9] = float("nan"), float("inf")
    _check(x, 5, renormalize=True)
    assert B.muon_query_status() == 7        # MUON_ERR_NONFINITE
    assert B.muon_query_status() == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("experts,k", [(1, 1), (7, 3), (64, 8), (130, 32), (256, 8), (1024, 4)])
def test_gradient(score, renorm, experts, k):
    for dtype in (F32, BF16):
        x = torch.randn(50, experts, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
        x[3, 0] = -float("inf")
        r, c = B.muon_route_forward(x, cfg := B.make_route_config(
            experts, k, score=NAMES[score], renormalize=renorm, scale=2.5)), cfg
        idx = r.idx.clone()
        idx[5] = -1
        idx[6, 0] = experts + 3              # out of range: reads as none
        dw = torch.randn(50, k, generator=torch.Generator().manual_seed(2)).cuda()
        got = _np(B.muon_route_backward(x, c, idx, dw))
        want = R.route_grad_ref(_np(x), idx.cpu().numpy(), _np(dw), score, renorm, 2.5)
        # sums over the row cancel: errors are relative to the terms' size
        size = 2.5 * np.abs(_np(dw)).max(1, keepdims=True)
        tol = 4e-6 * size + (2.0 ** -8 * np.abs(want) if dtype == BF16 else 0)
        if renorm:
            tol = tol * (1 + 1 / np.maximum(np.abs(_np(r.weights)).min(1, keepdims=True), 1e-3))
        assert np.all(np.abs(got - want) <= tol)
        assert np.all(got[5] == 0)


def test_gradient_is_the_difference_quotient():
    # a step of 1e-2: third derivative 1e-4, rounding 1e-7 / 1e-2; 2e-3 is held
    x, d = (torch.randn(200, 32, generator=torch.Generator().manual_seed(s)).cuda() for s in (1, 2))
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            c = B.make_route_config(32, 32, score=NAMES[score], renormalize=renorm)   # all: a fixed choice
            r = B.muon_route_forward(x, c)
            dw = torch.randn(200, 32, generator=torch.Generator().manual_seed(3)).cuda()
            by_expert = torch.zeros_like(dw).scatter_(1, r.idx.long(), dw)
            def f(v):
                q = B.muon_route_forward(v, c)
                return (by_expert.gather(1, q.idx.long()).double() * q.weights.double()).sum(1)
            slope = (f(x + 1e-2 * d) - f(x - 1e-2 * d)) / 2e-2
            got = (B.muon_route_backward(x, c, r.idx, dw).double() * d.double()).sum(1)
            assert float((got - slope).norm()) <= 2e-3 * float(slope.norm()) + 1e-6


def test_strides_plan_alone_and_no_tokens():
    x = torch.randn(30, 80, generator=torch.Generator().manual_seed(4)).cuda()
    c = B.make_route_config(50, 4)
    view = x[:, 7:57]
    a, b = B.muon_route_forward(view, c), B.muon_route_forward(view.contiguous(), c)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    dw = torch.randn(30, 4).cuda()
    out = torch.full((30, 60), 7.0, device="cuda")
    B.muon_route_backward(view, c, a.idx, dw, dlogits=out[:, 5:55])
    assert torch.equal(out[:, 5:55], B.muon_route_backward(view.contiguous(), c, a.idx, dw))
    assert bool((out[:, :5] == 7).all()) and bool((out[:, 55:] == 7).all())
    off, src, pos = B.muon_route_plan(a.idx, 50)
    assert torch.equal(off, a.offsets) and torch.equal(src, a.src) and torch.equal(pos, a.pos)
    assert B.muon_route_forward(view, c, plan=False).offsets is None
    e = B.muon_route_forward(torch.empty((0, 50), device="cuda"), c)
    assert e.idx.shape == (0, 4) and bool((e.offsets == 0).all())


def test_plan_reads_wild_indices_as_none():
    idx = torch.tensor([[5, -7], [1 << 30, 0], [4, 5]], dtype=torch.int32, device="cuda")
    off, src, pos = B.muon_route_plan(idx, 5)
    assert off.tolist() == [0, 1, 1, 1, 1, 2] and src.tolist() == [3, 4, -1, -1, -1, -1]
    assert pos.tolist() == [[-1, -1], [-1, 0], [1, -1]]
