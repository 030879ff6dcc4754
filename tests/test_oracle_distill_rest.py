"""Pins of the distillation oracle where the unlisted entries' share is far below a float's range (no GPU needed)."""
import math

import numpy as np
import pytest

from oracle import target_pass as O


def test_worked_rows():
    """One listed entry; s_R in closed form."""
    loss, grad, _ = O.distill([0.0, -9.0, -9.5, -10.0], [0], [0.0], 0.1, -math.log(0.9))
    tail = 1 + math.exp(-5) + math.exp(-10)
    assert abs(loss - (0.9 * math.log(0.9) + 0.1 * (math.log(0.1) + 90 - math.log(tail)))) < 1e-12
    assert np.allclose(grad, [1, -1 / tail, -math.exp(-5) / tail, -math.exp(-10) / tail], rtol=1e-12)
    # 10^7 nats below: nothing of s_R is left in float64
    loss, grad, parts = O.distill([0.0, -10.0, -10.0], [0], [0.0], 1e-6, -math.log(0.75))
    assert parts["s_rest"] == 0 and abs(loss / (0.25 * 1e7) - 1) < 1e-6
    assert np.allclose(grad, np.array([0.25, -0.125, -0.125]) * 1e6, rtol=1e-12)
    # at float32's lowest value, beside which a logarithm of their number is nothing: equal shares of p_R
    loss, grad, _ = O.distill([1.0] + [float(np.finfo(np.float32).min)] * 4, [0], [0.0], 1.0, -math.log(0.75))
    assert abs(loss / (0.25 * 3.4028234663852886e38) - 1) < 1e-12 and np.allclose(grad, [0.25] + [-0.0625] * 4, rtol=1e-12)
    # at -inf s_R is 0: the rest counts for nothing
    loss, grad, parts = O.distill([0.0, -math.inf], [0], [0.0], 1.0, math.log(2))
    assert parts["p_rest"] == 0 and abs(loss - 0.5 * math.log(0.5)) < 1e-15 and not grad.any()


@pytest.mark.parametrize("gap", [30.0, 90.0, 700.0, 1e4])
def test_gradient_is_the_losss_difference(gap):
    rng = np.random.default_rng(int(gap))
    V, tau = 11, 0.5
    x = rng.normal(size=V) - gap * tau
    ids, t = np.array([3, 7]), np.array([0.2, -0.4])
    x[ids] += gap * tau
    lse = math.log(np.exp(t / tau).sum() / 0.6)
    loss, grad, _ = O.distill(x, ids, t, tau, lse)
    assert abs(grad.sum()) < 1e-12
    e = 2.0 ** -12
    for v in range(V):
        step = np.eye(V)[v] * e
        d = (O.distill(x + step, ids, t, tau, lse)[0] - O.distill(x - step, ids, t, tau, lse)[0]) / (2 * e)
        # central differences: e^2 / 6 times a third derivative below 8 / tau^3, and a few 2^-52 |loss| / e of rounding
        assert abs(d - grad[v]) < 2 * e ** 2 / tau ** 3 + 2.0 ** -49 * (1 + abs(loss)) / e
