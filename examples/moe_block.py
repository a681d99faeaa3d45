"""A mixture-of-experts block trained with the library from end to end.

    python examples/moe_block.py [--steps 30] [--tokens 4096] [--hidden 1024]
                                 [--inner 512] [--experts 32] [--top-k 4]

One block h = x + r, y = norm(h), out = h + experts(y; route(y W_r^T)) fits a
random target.  Per step: RMS norm with the residual's addition, routing with
a balance bias, the experts' products and the gradients of all three; then Muon on
the experts' weights ([E, M, N] tensors, as the gradients come) and AdamW on
the gain and the router's weight.  The router's own product is a plain torch
matrix product.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from newton_schulz_gb300 import binding as B  # noqa: E402

EPS = 1e-6


class Block:
    def __init__(self, hidden, inner, experts, top_k, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        def randn(*shape, scale):
            return torch.randn(*shape, generator=gen, device=device).mul_(scale)
        self.gain = torch.ones(hidden, device=device)
        self.router = randn(experts, hidden, scale=hidden ** -0.5)
        self.w_in = randn(experts, 2 * inner, hidden, scale=hidden ** -0.5).bfloat16()
        self.w_out = randn(experts, hidden, inner, scale=inner ** -0.5).bfloat16()
        self.bias = torch.zeros(experts, device=device)      # moves with the load, not by gradient
        self.cfg = B.make_route_config(experts, top_k, score=B.ROUTE_SIGMOID, renormalize=True)
        self.mom_in = torch.zeros(self.w_in.shape, device=device)
        self.mom_out = torch.zeros(self.w_out.shape, device=device)
        self.adam = [[torch.zeros_like(t), torch.zeros_like(t)] for t in (self.gain, self.router)]
        self.steps = 0

    def forward(self, x, residual):
        y, h, _ = B.muon_rmsnorm_forward(x, self.gain, residual=residual, eps=EPS)
        logits = y.float() @ self.router.t()
        route = B.muon_route_forward(logits, self.cfg, bias=self.bias)
        out, gu = B.muon_experts_forward(y, self.w_in, self.w_out, route, save=True)
        return h.float() + out.float(), (y, h, logits, route, gu)

    def backward(self, grad, saved):
        """Gradients of the parameters and of x (and the residual) from that of the output."""
        y, h, logits, route, gu = saved
        grad = grad.bfloat16()
        dy, dw_in, dw_out, dweights = B.muon_experts_backward(grad, y, self.w_in, self.w_out, route, gu,
                                                              dw_dtype=torch.bfloat16)
        dlogits = B.muon_route_backward(logits, self.cfg, route.idx, dweights)
        drouter = dlogits.t() @ y.float()
        dy = (dy.float() + dlogits @ self.router).bfloat16()
        dx, dgain = B.muon_rmsnorm_backward(dy, h, self.gain, dres=grad, eps=EPS)
        return dict(x=dx, gain=dgain, router=drouter, w_in=dw_in, w_out=dw_out)

    def step(self, grads, route, lr=0.02, balance=1e-3):
        self.steps += 1
        e, two_i, hidden = self.w_in.shape
        halves = (2 * e, two_i // 2, hidden)      # gate and up matrices, each whole
        B.muon_step_grouped([
            dict(W=self.w_in.view(halves), G=grads["w_in"].view(halves), Mom=self.mom_in.view(halves)),
            dict(W=self.w_out, G=grads["w_out"], Mom=self.mom_out)], lr=lr, wd=0.0)
        B.muon_adamw_grouped([
            dict(param=p, grad=grads[n], exp_avg=s[0], exp_avg_sq=s[1])
            for n, p, s in zip(("gain", "router"), (self.gain, self.router), self.adam)],
            step=self.steps, lr=1e-3, weight_decay=0.0)
        load = route.offsets.diff().float()
        self.bias += balance * torch.sign(load.mean() - load)


def train(steps=30, tokens=4096, hidden=1024, inner=512, experts=32, top_k=4, seed=0, log=print):
    """Losses of `steps` steps."""
    block = Block(hidden, inner, experts, top_k, seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    x, residual, target = (torch.randn(tokens, hidden, generator=gen, device="cuda").bfloat16()
                           for _ in range(3))
    losses = []
    for k in range(steps):
        out, saved = block.forward(x, residual)
        diff = out - target.float()
        losses.append(float(diff.square().mean()))
        block.step(block.backward(diff * (2.0 / diff.numel()) * tokens, saved), saved[3])
        if k % 10 == 0 or k + 1 == steps:
            load = saved[3].offsets.diff().float()
            log(f"step {k:3d}  loss {losses[-1]:.4f}  busiest expert {float(load.max() / load.mean()):.2f}x the mean")
    status = B.muon_query_status()
    if status != B.MUON_OK:
        raise RuntimeError(B.muon_status_string(status))
    return losses


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    for name, value in (("steps", 30), ("tokens", 4096), ("hidden", 1024), ("inner", 512), ("experts", 32),
                        ("top-k", 4)):
        p.add_argument("--" + name, type=int, default=value)
    train(**{k.replace("-", "_"): v for k, v in vars(p.parse_args()).items()})
