"""One small case for every kernel of the mixture-of-experts block, run through
whichever libmuon the process loads (MUON_LIB_PATH selects the -DMUON_DEBUG
build), as debug_cases.py does for the optimizer's.

    python tests/debug_block_cases.py OUT.npz
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from newton_schulz_gb300 import binding as B  # noqa: E402

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


def _randn(*shape, dtype=BF16, seed=1):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def main(out_path):
    B.load()
    res, codes = {}, {}

    def keep(name, outs):
        torch.cuda.synchronize()
        codes[name] = B.muon_query_status()
        for i, t in enumerate(outs):
            if t is not None:
                res[f"{name}.{i}"] = t.float().cpu().numpy()

    # every chunk count of the norm's kernels, both widths; ragged, unaligned
    for rows, cols, dt in ((3, 4096, BF16), (700, 2048, F32), (700, 4096, BF16), (700, 12000, BF16), (5, 9, F32),
                           (700, 12001, F32)):
        x, r, g = _randn(rows, cols, dtype=dt), _randn(rows, cols, dtype=dt, seed=2), _randn(cols, seed=3)
        keep(f"norm {rows} {cols}", B.muon_rmsnorm_forward(x, g, residual=r))
        keep(f"norm gradient {rows} {cols}", B.muon_rmsnorm_backward(x, r, g, dres=r))
    for group in (0, 128):
        keep(f"e4m3 {group}", B.muon_rmsnorm_forward(_randn(50, 1000), y_dtype=E4M3, group=group))
    for cols in (2048, 8192):
        x = _randn(1500, cols)
        keep(f"ring {cols}", B.muon_rmsnorm_backward(x, _randn(1500, cols, seed=2), _randn(cols, seed=3), dres=x))
    # every number of experts a lane, grouped and not; one and several tiles of the plan
    for experts in (7, 64, 100, 256, 500, 1024):
        for tokens in (33, 600):
            logits = _randn(tokens, experts, dtype=F32, seed=experts)
            groups = 1 if experts in (7, 500) else 4
            cfg = B.make_route_config(experts, 4, score=B.ROUTE_SIGMOID, groups=groups, top_groups=max(1, groups // 2),
                                      renormalize=True)
            r = B.muon_route_forward(logits, cfg, mask=torch.arange(tokens, device="cuda") % 5 > 0)
            keep(f"route {experts} {tokens}", r)
            keep(f"plan {experts} {tokens}", B.muon_route_plan(r.idx, experts))
            keep(f"route gradient {experts} {tokens}",
                 [B.muon_route_backward(logits, cfg, r.idx, _randn(tokens, 4, dtype=F32))])
    # the products: a few rows, one pair, clusters of two, repacked weights, the copy beside dx
    for tokens, k, hidden, inner, experts in ((5, 3, 200, 136, 9), (5, 3, 131, 77, 9), (300, 2, 264, 136, 5),
                                              (90, 2, 131, 77, 5), (1100, 1, 1024, 1032, 3), (8300, 2, 512, 512, 4)):
        idx = torch.rand(tokens, experts, generator=torch.Generator().manual_seed(1)).argsort(1)[:, :k]
        idx = torch.where(torch.rand(tokens, k, generator=torch.Generator().manual_seed(2)) < 0.05, -1, idx)
        idx = idx.to(torch.int32).cuda()
        r = B.Route(idx, _randn(tokens, k, dtype=F32).abs(), *B.muon_route_plan(idx, experts))
        x, dout = _randn(tokens, hidden), _randn(tokens, hidden, seed=2)
        w_in = _randn(experts, 2 * inner, hidden, seed=3) * hidden ** -0.5
        w_out = _randn(experts, hidden, inner, seed=4) * inner ** -0.5
        out, gu = B.muon_experts_forward(x, w_in, w_out, r, save=True)
        name = f"experts {tokens} {hidden} {inner}"
        keep(name, (out, gu[:int(r.offsets[-1])]))
        for dt in (F32, BF16):
            keep(f"{name} gradient {dt}", B.muon_experts_backward(dout, x, w_in, w_out, r, gu, dw_dtype=dt))

    np.savez(out_path, codes=np.array([codes[k] for k in sorted(codes)]),
             names=np.array(sorted(codes)), debug_build=np.array(B.muon_debug_build()), **res)


if __name__ == "__main__":
    main(sys.argv[1])
