"""The mixture-of-experts oracle's gradients against central differences of
its forward functions, in float64 (CPU).  A central difference of step 1e-6
of these smooth functions of order one errs by about 1e-12 (truncation)
+ 1e-10 (cancellation); 1e-7 relative is held."""
import numpy as np
import pytest

from oracle import moe_ref as R


def _slope(f, x, d, step=1e-6):
    return (f(x + step * d) - f(x - step * d)) / (2 * step)


@pytest.mark.parametrize("gain", [True, False])
def test_rmsnorm_gradient_is_the_difference_quotient(gain):
    r = np.random.default_rng(1)
    h, dy, d = (r.standard_normal((3, 17)) for _ in range(3))
    g = 1 + 0.1 * r.standard_normal(17) if gain else None
    dh, dgain = R.rmsnorm_grad_ref(dy, h, g, None, 1e-3)
    f = lambda v: float((dy * R.rmsnorm_ref(v, None, g, 1e-3)[1]).sum())  # noqa: E731
    assert abs(float((dh * d).sum()) - _slope(f, h, d)) <= 1e-7 * np.linalg.norm(dh) * np.linalg.norm(d)
    if gain:
        q = lambda v: float((dy * R.rmsnorm_ref(h, None, v, 1e-3)[1]).sum())  # noqa: E731
        assert abs(float((dgain * d[0]).sum()) - _slope(q, g, d[0])) <= 1e-7 * np.linalg.norm(dgain) * 10


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_is_the_difference_quotient(score, renorm):
    r = np.random.default_rng(2)
    x, d = r.standard_normal((5, 12)), r.standard_normal((5, 12))
    idx, _ = R.route_ref(x, 3, score=score, renormalize=renorm)
    idx[1, 2] = -1
    dw = r.standard_normal(idx.shape)
    grad = R.route_grad_ref(x, idx, dw, score, renorm, 2.5)
    f = lambda v: float((dw * R.route_weights_ref(v, idx, score, renorm, 2.5)).sum())  # noqa: E731
    assert abs(float((grad * d).sum()) - _slope(f, x, d)) <= 1e-7 * np.linalg.norm(grad) * np.linalg.norm(d)


def test_experts_gradient_is_the_difference_quotient():
    r = np.random.default_rng(3)
    E, H, I, T, k = 3, 6, 5, 4, 2
    x, w_in, w_out = r.standard_normal((T, H)), r.standard_normal((E, 2 * I, H)), r.standard_normal((E, H, I))
    idx = np.array([[0, 2], [1, -1], [2, 0], [1, 2]])
    w, dout = r.standard_normal((T, k)), r.standard_normal((T, H))
    _, gu = R.experts_ref(x, w_in, w_out, idx, w)
    grads = R.experts_grad_ref(dout, x, w_in, w_out, idx, w, gu)
    args = [x, w_in, w_out, w]
    for i in range(4):
        def f(v):
            a = list(args)
            a[i] = v
            return float((dout * R.experts_ref(a[0], a[1], a[2], idx, a[3])[0]).sum())
        d = r.standard_normal(args[i].shape)
        got = float((grads[i] * d).sum())
        assert abs(got - _slope(f, args[i], d)) <= 1e-7 * np.linalg.norm(grads[i]) * np.linalg.norm(d)


def test_route_rules():
    inf = np.inf
    # ties to the lowest index; -inf and NaN never chosen; empty slots
    idx, w = R.route_ref(np.array([[1.0, 2.0, 2.0, 0.0], [-inf, 3.0, -inf, -inf], [-inf] * 4,
                                   [np.nan, 1.0, 1.0, inf]]), 2)
    assert idx.tolist() == [[1, 2], [1, -1], [-1, -1], [1, 2]]
    assert w[1].tolist() == [1.0, 0.0] and w[2].tolist() == [0.0, 0.0]
    # the bias moves the choice, not the weight
    idx, w = R.route_ref(np.zeros((1, 3)), 1, score="sigmoid", bias=np.array([0.0, 0.0, 0.1]))
    assert idx.tolist() == [[2]] and w.tolist() == [[0.5]]
    # groups by their two best: 0.9 alone loses to 0.6 + 0.6
    p = np.array([0.9, 0.1, 0.6, 0.6])
    idx, _ = R.route_ref(np.log(p / (1 - p))[None], 1, score="sigmoid", groups=2, top_groups=1,
                         group_score="sum2")
    assert idx.tolist() == [[2]]


def test_plan_is_a_stable_sort():
    off, src, pos = R.plan_ref(np.array([[2, 0], [-1, 2], [0, 2]]), 4)
    assert off.tolist() == [0, 2, 2, 5, 5]
    assert src.tolist() == [1, 4, 0, 3, 5, -1]
    assert pos.tolist() == [[2, 0], [-1, 3], [1, 4]]
