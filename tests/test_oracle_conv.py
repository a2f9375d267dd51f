"""Pins of the convolution oracle: a hand-worked example, the split at any token, and its
gradients against central differences. Runs on the CPU."""

import numpy as np
import pytest

from oracle import conv, conv_bwd


def test_hand_worked():
    x = np.array([[1.0], [2.0], [-1.0]])
    w = np.array([[0.5, -1.0, 2.0]])
    y, final = conv(x, w, np.array([0.25]), silu=False)
    # taps reach back two rows; rows before the first are zero
    assert np.allclose(y[:, 0], [0.25 + 2, 0.25 - 1 + 4, 0.25 + 0.5 - 2 - 2])
    assert np.array_equal(final[:, 0], [2.0, -1.0])
    y, final = conv(x[:1], w, None, np.array([[3.0], [4.0]]), silu=False)
    assert np.allclose(y[:, 0], [1.5 - 4 + 2]) and np.array_equal(final[:, 0], [4.0, 1.0])
    y, _ = conv(x, w, np.array([0.25]))
    assert np.allclose(y[0, 0], 2.25 / (1 + np.exp(-2.25)))


@pytest.mark.parametrize("W", [2, 3, 4])
def test_split_anywhere(W):
    rng = np.random.default_rng(W)
    x, w, b = rng.normal(size=(9, 5)), rng.normal(size=(5, W)), rng.normal(size=5)
    s0 = rng.normal(size=(W - 1, 5))
    y, final = conv(x, w, b, s0)
    for cut in range(10):
        y1, s1 = conv(x[:cut], w, b, s0)
        y2, s2 = conv(x[cut:], w, b, s1)
        assert np.allclose(np.concatenate([y1, y2]), y) and np.array_equal(s2, final)


@pytest.mark.parametrize("T,W,silu", [(5, 4, True), (1, 4, True), (2, 3, False), (0, 3, True)])
def test_gradients_against_differences(T, W, silu):
    rng = np.random.default_rng(10 * T + W)
    D = 2
    a = dict(x=rng.normal(size=(T, D)), weight=rng.normal(size=(D, W)), bias=rng.normal(size=D),
             state=rng.normal(size=(W - 1, D)))
    dy, df = rng.normal(size=(T, D)), rng.normal(size=(W - 1, D))
    dx, dw, db, ds = conv_bwd(a["x"], a["weight"], dy, a["bias"], a["state"], df, silu)[0]

    def loss(**kw):
        y, f = conv(**dict(a, **kw), silu=silu)
        return float((y * dy).sum() + (f * df).sum())

    eps = 1e-6
    for name, got in (("x", dx), ("weight", dw), ("bias", db), ("state", ds)):
        for i in np.ndindex(*a[name].shape):
            up, down = a[name].copy(), a[name].copy()
            up[i] += eps
            down[i] -= eps
            diff = (loss(**{name: up}) - loss(**{name: down})) / (2 * eps)
            # central differences: eps^2 |f'''| / 6 plus rounding 2^-53 |f| / eps, both under 1e-8 here
            assert abs(diff - got[i]) <= 1e-6 * max(1.0, abs(diff)), (name, i)
