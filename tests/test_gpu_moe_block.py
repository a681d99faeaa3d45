"""The mixture-of-experts block as a program uses it: the example trains, and
its gradients agree with automatic differentiation of the same block written
in plain torch (float64, the routing's choice held fixed).  The block rounds
activations and gradients to bf16 at five places on the longest path (2^-8 / sqrt 3
each, independent): 5e-3, held to 1e-2 in norm."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")


@pytest.fixture(scope="module")
def example(lib, cuda_ok):
    spec = importlib.util.spec_from_file_location("moe_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_trains(example):
    losses = example.train(steps=12, tokens=600, hidden=192, inner=136, experts=6, top_k=2, log=lambda s: None)
    assert losses[-1] < 0.9 * losses[0]


def test_gradients_agree_with_automatic_differentiation(example):
    block = example.Block(160, 72, 5, 2, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, r = (torch.randn(200, 160, generator=gen, device="cuda").bfloat16() for _ in range(2))
    grad = torch.randn(200, 160, generator=gen, device="cuda").bfloat16()
    out, saved = block.forward(x, r)
    got = block.backward(grad, saved)
    par = {n: getattr(block, n).double().requires_grad_(True) for n in ("gain", "router", "w_in", "w_out")}
    xd = x.double().requires_grad_(True)
    h = xd + r.double()
    y = par["gain"] * h / torch.sqrt((h * h).mean(1, keepdim=True) + example.EPS)
    idx = saved[3].idx.long()
    score = torch.sigmoid(y @ par["router"].t()).gather(1, idx)
    w = score / score.sum(1, keepdim=True)
    res = h
    for j in range(2):
        gate, up = torch.einsum("tfh,th->tf", par["w_in"][idx[:, j]], y).chunk(2, 1)
        act = gate * torch.sigmoid(gate) * up
        res = res + w[:, j:j + 1] * torch.einsum("thi,ti->th", par["w_out"][idx[:, j]], act)
    res.backward(grad.double())
    assert float((out.double() - res).norm()) <= 1e-2 * float(res.norm())
    for n, want in (("x", xd.grad), *((k, v.grad) for k, v in par.items())):
        assert float((got[n].double() - want).norm()) <= 1e-2 * float(want.norm()), n
