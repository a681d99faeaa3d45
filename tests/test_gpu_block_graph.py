"""The block's calls in a CUDA graph: a decode step (norm, routing, experts)
captured on a stream that has no workspace yet, run again with other inputs, and
again after a larger call on the capturing stream has outgrown the workspace that
the graph names."""
import pytest
import torch

from newton_schulz_gb300 import binding as B

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
HIDDEN, INNER, EXPERTS, TOP_K = 256, 136, 16, 4


@pytest.fixture(autouse=True)
def _dev(lib, cuda_ok):
    yield
    torch.cuda.synchronize()
    assert B.muon_query_status() == 0


def _randn(*shape, dtype=BF16, seed=1):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


class Weights:
    def __init__(self):
        self.gain = _randn(HIDDEN, seed=3)
        self.router = _randn(EXPERTS, HIDDEN, dtype=F32, seed=4) * HIDDEN ** -0.5
        self.w_in = _randn(EXPERTS, 2 * INNER, HIDDEN, seed=5) * HIDDEN ** -0.5
        self.w_out = _randn(EXPERTS, HIDDEN, INNER, seed=6) * INNER ** -0.5
        self.cfg = B.make_route_config(EXPERTS, TOP_K, renormalize=True)

    def step(self, x, res):
        y, h, _ = B.muon_rmsnorm_forward(x, self.gain, residual=res)
        r = B.muon_route_forward((y.float()[:, None, :] * self.router).sum(2), self.cfg)
        return h, r.idx, B.muon_experts_forward(y, self.w_in, self.w_out, r)[0]

    def train(self, x, dout):
        idx = torch.arange(x.shape[0], dtype=torch.int32, device="cuda")[:, None] % EXPERTS
        r = B.Route(idx, torch.ones(x.shape[0], 1, device="cuda"), *B.muon_route_plan(idx, EXPERTS))
        out, gu = B.muon_experts_forward(x, self.w_in, self.w_out, r, save=True)
        return (out, *B.muon_experts_backward(dout, x, self.w_in, self.w_out, r, gu),
                *B.muon_rmsnorm_backward(dout, x, self.gain))


@pytest.mark.parametrize("tokens", [1, 8, 40, 600])      # 600: the row plan's counts need a workspace
def test_decode_step(tokens):
    w = Weights()
    x, res = _randn(tokens, HIDDEN, seed=7), _randn(tokens, HIDDEN, seed=8)
    w.step(x, res)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = w.step(x, res)
    for seed in (10, 20):
        x.copy_(_randn(tokens, HIDDEN, seed=seed))
        res.copy_(_randn(tokens, HIDDEN, seed=seed + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, w.step(x, res)))
    # outgrow the workspace on that stream, and let others take memory
    big, dout = _randn(5000, HIDDEN, seed=30), _randn(5000, HIDDEN, seed=31)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        first = w.train(big, dout)
    torch.cuda.synchronize()
    junk = [torch.full((1 << 21,), float("nan"), device="cuda") for _ in range(16)]
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, w.step(x, res)))
    with torch.cuda.stream(side):
        again = w.train(big, dout)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    del junk


def test_training_calls():
    w = Weights()
    x, dout = _randn(300, HIDDEN, seed=7), _randn(300, HIDDEN, seed=8)
    w.train(x, dout)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        got = w.train(x, dout)
    x.copy_(_randn(300, HIDDEN, seed=9))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, w.train(x, dout)))


def test_gradient_through_clusters_and_copies_beside(monkeypatch):
    # 16500 rows over 16 experts, K of 1024: the launch forms of a training batch
    import sys
    m = sys.modules[__name__]
    monkeypatch.setattr(m, "HIDDEN", 1024)
    monkeypatch.setattr(m, "INNER", 520)
    w = Weights()
    x, dout = _randn(16500, 1024, seed=7), _randn(16500, 1024, seed=8)
    w.train(x, dout)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        got = w.train(x, dout)
    x.copy_(_randn(16500, 1024, seed=9))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, w.train(x, dout)))
