"""Routing scores where an exponential is large or small.

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
