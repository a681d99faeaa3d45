"""Routing scores and their gradients where an exponential is large or small.

Tolerances: an exponential (2 units of the last place), a quotient (2) and at
most three products (half a unit each) are under 8 * 2^-24 = 5e-7 of the
value; sums of at most 8 like terms add 8 * 2^-24.  Below 2^-126 a unit of the
last place is 2^-149: an exponential and a product there may err by 2^-148.
2e-6 relative is held, 4e-6 where a sum of scores divides."""
import numpy as np
import pytest
import torch

from newton_schulz_gb300 import binding as B
from oracle import moe_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _dev(lib, cuda_ok):
    yield


def _np(t):
    return t.detach().double().cpu().numpy()


def test_sigmoid_gradient_of_large_logits():
    # s (1 - s): 1 - s is 4e-8 at 17 and below half a unit of s's last place there
    x = torch.tensor([[a, -a, b, -b] for a in (8.0, 10.0, 12.0, 14.5) for b in (16.0, 17.5, 20.0, 40.0, 80.0)],
                     device="cuda")
    cfg = B.make_route_config(4, 4, score=B.ROUTE_SIGMOID)
    r = B.muon_route_forward(x, cfg)
    dw = torch.randn(x.shape[0], 4, generator=torch.Generator().manual_seed(1)).cuda()
    got = _np(B.muon_route_backward(x, cfg, r.idx, dw))
    l, d = _np(x), np.zeros(x.shape)
    np.put_along_axis(d, r.idx.cpu().numpy().astype(np.int64), _np(dw), 1)
    want = d / (1 + np.exp(-l)) / (1 + np.exp(l))
    assert np.all(np.abs(got - want) <= 2e-6 * np.abs(want) + 2.0 ** -149)


def test_sigmoid_weights_of_very_low_logits():
    # scores near and below the least normal number still have a ratio
    x = torch.tensor([[-87.0, -87.5, -88.0, -88.5], [-88.6, -87.4, -88.1, -87.9], [-87.5, -90.0, -60.0, -87.6]],
                     device="cuda")
    cfg = B.make_route_config(4, 3, score=B.ROUTE_SIGMOID, renormalize=True)
    r = B.muon_route_forward(x, cfg)
    idx, w = R.route_ref(_np(x), 3, score="sigmoid", renormalize=True)
    assert np.array_equal(r.idx.cpu().numpy(), idx)
    assert np.all(np.abs(_np(r.weights) - w) <= 4e-6 * w)
    plain = B.muon_route_forward(x, B.make_route_config(4, 3, score=B.ROUTE_SIGMOID)).weights
    s = np.take_along_axis(1 / (1 + np.exp(-_np(x))), idx, 1)
    assert np.all(np.abs(_np(plain) - s) <= 2e-6 * s + 2.0 ** -148)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_renormalised_gradient_of_small_scores(score):
    # a bias sends a token to experts whose scores are tiny; the gradient is of
    # the weights' size times 1 - s, whatever the scores' sum
    x = torch.tensor([[0.0, -85.0, -86.0, -86.5], [0.0, -86.9, -84.0, -85.5]], device="cuda")
    bias = torch.tensor([-2.0, 1.0, 1.5, 2.0], device="cuda")
    cfg = B.make_route_config(4, 3, score=getattr(B, "ROUTE_" + score.upper()), renormalize=True, scale=2.5)
    r = B.muon_route_forward(x, cfg, bias=bias)
    assert r.idx.tolist() == [[3, 2, 1]] * 2
    dw = torch.tensor([[120.0, -80.0, 55.0], [-90.0, 70.0, 100.0]], device="cuda")
    got = _np(B.muon_route_backward(x, cfg, r.idx, dw))
    l, w = _np(x), _np(dw)
    want = np.zeros_like(l)
    for t in range(2):
        at = r.idx[t].tolist()
        q = np.exp(l[t, at])
        q /= q.sum()
        want[t, at] = 2.5 * q * (w[t] - (w[t] * q).sum())
    # (the sigmoid's 1 - s and the softmax's rest are 1 to 64 bits here)
    assert np.all(np.abs(got - want) <= 4e-6 * 2.5 * np.abs(w).max(1, keepdims=True))
