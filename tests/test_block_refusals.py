"""Refusals of the mixture-of-experts block's entry points: bad arguments are
rejected on the host before anything touches CUDA (no device needed), with
the code that include/muon.h names."""
import ctypes

import pytest

from newton_schulz_gb300 import binding as B

INV, UNS, ALIAS = 1, 2, 3
P = 0x10000000          # stand-in device addresses, far apart, never read


def _at(i):
    return P + (i << 32)


def _norm(**kw):
    a = B.RmsNorm(rows=4, cols=64, x=_at(0), x_stride=64, y=_at(1), y_stride=64, x_dtype=1, y_dtype=1,
                  eps=1e-6)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INV), (dict(cols=-1), INV), (dict(x=None), INV), (dict(y=None), INV),
    (dict(x_dtype=2), INV), (dict(x_dtype=7), INV), (dict(y_dtype=3), INV), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(x_stride=63), INV), (dict(y_stride=1), INV),
    (dict(group=128), INV), (dict(y_dtype=2), INV), (dict(y_dtype=2, scales=_at(2), group=64), INV),
    (dict(x=_at(0) + 1), INV), (dict(cols=32769, x_stride=40000, y_stride=40000), UNS),
    (dict(rows=1 << 31), UNS), (dict(y=_at(0)), ALIAS), (dict(y=_at(0) + 128), ALIAS),
    (dict(residual=_at(3), residual_dtype=2, residual_stride=64), INV),
    (dict(residual=_at(3), residual_dtype=1, residual_stride=64, h=_at(3), h_dtype=0, h_stride=64), ALIAS),
    (dict(residual=_at(3), residual_dtype=1, residual_stride=64, h=_at(3) + 2, h_dtype=1, h_stride=64),
     ALIAS),
    (dict(h=_at(1), h_dtype=1, h_stride=64), ALIAS), (dict(gain=_at(1), gain_dtype=1), ALIAS),
    (dict(y_dtype=2, scales=_at(1)), ALIAS)])
def test_rmsnorm_forward_refuses(lib, kw, code):
    assert lib.muon_rmsnorm_forward(ctypes.byref(_norm(**kw)), None) == code


def test_null_argument_structures(lib):
    assert lib.muon_rmsnorm_forward(None, None) == INV
    assert lib.muon_rmsnorm_backward(None, None) == INV
    assert lib.muon_experts_forward(None, None, 0, None, None) == INV
    assert lib.muon_experts_backward(None, None, 0, None, None, 0, None, None, 0, None, None) == INV
    assert lib.muon_route_forward(None, P, 0, 8, 1, None, None, P, P, None, None, None, None) == INV
    assert lib.muon_route_backward(None, P, 0, 8, 1, P, P, P, 8, None) == INV


def test_no_rows_is_a_no_op(lib):
    assert lib.muon_rmsnorm_forward(ctypes.byref(_norm(rows=0, x=None, y=None)), None) == 0
    assert lib.muon_last_launch_count() == 0


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INV), (dict(dy=None), INV), (dict(h=None), INV), (dict(dh=None), INV),
    (dict(dy_dtype=2), INV), (dict(dh_dtype=2), INV), (dict(dy_stride=8), INV), (dict(eps=-1.0), INV),
    (dict(cols=32769), UNS), (dict(dgain=_at(4) + 2), INV), (dict(dh=_at(1)), ALIAS),
    (dict(dh=_at(0), dh_dtype=0), ALIAS), (dict(dgain=_at(0)), ALIAS), (dict(dgain=_at(2)), ALIAS)])
def test_rmsnorm_backward_refuses(lib, kw, code):
    a = B.RmsNormGrad(rows=4, cols=64, dy=_at(0), dy_stride=64, h=_at(1), h_stride=64, dh=_at(2),
                      dh_stride=64, dy_dtype=1, h_dtype=1, dh_dtype=1, eps=1e-6)
    for k, v in kw.items():
        setattr(a, k, v)
    assert lib.muon_rmsnorm_backward(ctypes.byref(a), None) == code


def _route(lib, cfg=None, logits=_at(0), dtype=0, stride=8, tokens=4, bias=None, mask=None, idx=_at(1),
           weights=_at(2), off=_at(3), src=_at(4), pos=_at(5)):
    cfg = cfg or B.make_route_config(8, 2)
    return lib.muon_route_forward(ctypes.byref(cfg), logits, dtype, stride, tokens, bias, mask, idx,
                                  weights, off, src, pos, None)


@pytest.mark.parametrize("cfg,code", [
    (dict(experts=0, top_k=1), INV), (dict(experts=8, top_k=0), INV), (dict(experts=8, top_k=9), INV),
    (dict(experts=8, top_k=2, score=2), INV), (dict(experts=8, top_k=2, groups=3), INV),
    (dict(experts=8, top_k=2, groups=0), INV), (dict(experts=8, top_k=2, groups=2, top_groups=3), INV),
    (dict(experts=8, top_k=2, groups=2, top_groups=0), INV), (dict(experts=8, top_k=2, group_score=2), INV),
    (dict(experts=8, top_k=2, scale=float("inf")), INV), (dict(experts=1025, top_k=2), UNS),
    (dict(experts=64, top_k=33), UNS), (dict(experts=130, top_k=2, groups=65), UNS)])
def test_route_config_refused(lib, cfg, code):
    assert _route(lib, B.make_route_config(**cfg), stride=2000) == code


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), INV), (dict(dtype=2), INV), (dict(stride=7), INV), (dict(logits=None), INV),
    (dict(idx=None), INV), (dict(weights=None), INV), (dict(src=None), INV), (dict(pos=None), INV),
    (dict(off=_at(3) + 1), INV), (dict(tokens=1 << 30), UNS), (dict(idx=_at(0)), ALIAS),
    (dict(src=_at(5)), ALIAS), (dict(bias=_at(2)), ALIAS), (dict(mask=_at(4)), ALIAS)])
def test_route_forward_refuses(lib, kw, code):
    assert _route(lib, **kw) == code


def test_route_backward_and_plan_refuse(lib):
    cfg = ctypes.byref(B.make_route_config(8, 2))
    f = lib.muon_route_backward
    assert f(cfg, _at(0), 2, 8, 4, _at(1), _at(2), _at(3), 8, None) == INV
    assert f(cfg, _at(0), 0, 8, 4, _at(1), _at(2), None, 8, None) == INV
    assert f(cfg, _at(0), 0, 8, 4, _at(1), _at(2), _at(3), 7, None) == INV
    assert f(cfg, _at(0), 0, 8, 4, _at(1), _at(2), _at(0), 8, None) == ALIAS
    g = lib.muon_route_plan
    assert g(_at(0), -1, 2, 8, _at(1), _at(2), _at(3), None) == INV
    assert g(_at(0), 4, 0, 8, _at(1), _at(2), _at(3), None) == INV
    assert g(None, 4, 2, 8, _at(1), _at(2), _at(3), None) == INV
    assert g(_at(0), 4, 2, 8, None, _at(2), _at(3), None) == INV
    assert g(_at(0), 4, 2, 1025, _at(1), _at(2), _at(3), None) == UNS
    assert g(_at(0), 4, 2, 8, _at(1), _at(2), _at(2), None) == ALIAS


def _experts(**kw):
    a = B.Experts(4, 64, 32, 8, 2, _at(0), 64, _at(1), _at(2), _at(3), _at(4), _at(5), _at(6))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), INV), (dict(hidden=0), INV), (dict(inner=0), INV), (dict(experts=0), INV),
    (dict(top_k=0), INV), (dict(x=None), INV), (dict(w_in=None), INV), (dict(w_out=None), INV),
    (dict(weights=None), INV), (dict(offsets=None), INV), (dict(src=None), INV), (dict(pos=None), INV),
    (dict(x_stride=63), INV), (dict(x=_at(0) + 1), INV), (dict(experts=1025), UNS), (dict(top_k=33), UNS),
    (dict(hidden=65537, x_stride=65537), UNS), (dict(inner=65537), UNS), (dict(tokens=1 << 30), UNS)])
def test_experts_refuse(lib, kw, code):
    a = ctypes.byref(_experts(**kw))
    stride = max(64, kw.get("hidden", 64))
    assert lib.muon_experts_forward(a, _at(7), stride, None, None) == code
    assert lib.muon_experts_backward(a, _at(8), stride, _at(9), _at(10), stride, _at(11), _at(12), 0, _at(13),
                                     None) == code


def test_experts_outputs_refused(lib):
    a = ctypes.byref(_experts())
    f, g = lib.muon_experts_forward, lib.muon_experts_backward
    assert f(a, None, 64, None, None) == INV
    assert f(a, _at(7), 63, None, None) == INV
    assert f(a, _at(7), 64, _at(8) + 1, None) == INV
    assert f(a, _at(0), 64, None, None) == ALIAS
    assert f(a, _at(7), 64, _at(7), None) == ALIAS
    ok = [a, _at(8), 64, _at(9), _at(10), 64, _at(11), _at(12), 0, _at(13), None]
    for i, v, code in ((1, None, INV), (3, None, INV), (2, 63, INV), (5, 63, INV), (8, 2, INV),
                       (4, _at(8), ALIAS), (6, _at(1), ALIAS), (7, _at(11), ALIAS), (9, _at(3), ALIAS)):
        bad = list(ok)
        bad[i] = v
        assert g(*bad) == code, i


def test_binding_refuses_wrong_tensors():
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        B.muon_rmsnorm_forward(x)                       # not on the device
    with pytest.raises(TypeError):
        B.muon_experts_forward(x, x, torch.zeros(2, 8, 4), B.Route(x, x, x, x, x))
    with pytest.raises(ValueError):
        B.muon_route_plan(torch.zeros(4, 2, dtype=torch.int64), 8)
