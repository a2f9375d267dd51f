"""Pins of the oracles of the norms, the gated linear recurrence and the checkpoints: hand-worked
values, invariants, and gradients against central differences. Runs on the CPU."""

import numpy as np
import pytest

from oracle import (checkpoint_pack, checkpoint_unpack, gate, glr, glr_bwd, glr_gates, postnorm, postnorm_bwd, prenorm,
                    prenorm_bwd)


def _differences(loss, args, grads, eps=1e-6):
    for name, got in grads.items():
        if got is None:
            continue
        for i in np.ndindex(*args[name].shape):
            up, down = args[name].copy(), args[name].copy()
            up[i] += eps
            down[i] -= eps
            diff = (loss(**{name: up}) - loss(**{name: down})) / (2 * eps)
            # central differences: eps^2 |f'''| / 6 plus rounding 2^-53 |f| / eps, both under 1e-8 here
            assert abs(diff - got[i]) <= 1e-6 * max(1.0, abs(diff)), (name, i, diff, got[i])


def test_norms_hand_worked():
    x, r = np.array([[3.0, 4.0]]), np.array([[1.0, -4.0]])
    y, h = prenorm(x, np.array([1.0, 2.0]), r, np.array([1.0, 2.0]), eps=2.0)
    assert np.allclose(h, [[4.0, 4.0]]) and np.allclose(y, [[4 / np.sqrt(18), 8 / np.sqrt(18)]])
    y = postnorm(x, np.array([1.0, 1.0]), np.array([[0.0, 1.0]]), r, np.array([2.0, 1.0]), eps=3.5)
    assert np.allclose(y, [[1 + 2 * 0.5 * 3 / 4, -4 + 4 / 4 / (1 + np.exp(-1.0))]])
    y = postnorm(x, np.array([1.0, 1.0]), np.array([[0.0, 1.0]]), silu=True, eps=3.5)
    assert np.allclose(y, [[0.0, 1 / (1 + np.exp(-1.0))]])


@pytest.mark.parametrize("residual,scale", [(True, True), (False, False), (True, False), (False, True)])
def test_prenorm_gradients(residual, scale):
    rng = np.random.default_rng(1)
    a = dict(x=rng.normal(size=(3, 5)), weight=rng.normal(size=5), residual=rng.normal(size=(3, 5)) if residual else None,
             scale=rng.normal(size=5) if scale else None)
    dy, dh = rng.normal(size=(3, 5)), rng.normal(size=(3, 5))

    def loss(**kw):
        y, h = prenorm(**dict(a, **kw))
        return float((y * dy).sum() + (h * dh).sum())

    dres, dx, dw, ds = prenorm_bwd(prenorm(**a)[1], a["weight"], dy, dh, a["x"], a["scale"])
    _differences(loss, a, dict(x=dx, weight=dw, scale=ds, residual=dres if residual else None))


@pytest.mark.parametrize("gate,scale,silu", [(True, True, False), (True, True, True), (False, False, False),
                                             (True, False, True)])
def test_postnorm_gradients(gate, scale, silu):
    rng = np.random.default_rng(2)
    a = dict(x=rng.normal(size=(2, 2, 4)), weight=rng.normal(size=4), gate=rng.normal(size=(2, 2, 4)) if gate else None,
             scale=rng.normal(size=4) if scale else None)
    dy = rng.normal(size=(2, 2, 4))
    dx, dg, dw, ds = postnorm_bwd(a["x"], a["weight"], dy, a["gate"], a["scale"], silu)
    _differences(lambda **kw: float((postnorm(**dict(a, **kw), silu=silu) * dy).sum()), a,
                 dict(x=dx, gate=dg, weight=dw, scale=ds))


def _glr_args(rng, T, D, in_gate=True, state=True):
    return dict(x=rng.normal(size=(T, D)), gate_x=rng.normal(size=(T, D)), A_log=0.3 * rng.normal(size=D),
                dt_bias=rng.normal(size=D), in_gate=rng.normal(size=(T, D)) if in_gate else None,
                state=rng.normal(size=D) if state else None)


def test_recurrence_hand_worked_and_its_gate():
    ln2 = np.log(2.0)
    # softplus(0) = ln 2: a rate of 2 gives the decay 1/4
    args = dict(x=np.array([[1.0], [2.0]]), gate_x=np.zeros((2, 1)), A_log=np.array([ln2]))
    y, h = glr(**args, state=np.array([8.0]), normalise=False)
    assert np.allclose(y[:, 0], [3.0, 2.75]) and np.allclose(h, [2.75])
    y, _ = glr(**args, in_gate=np.zeros((2, 1)))
    w = np.sqrt(1 - 1 / 16)
    assert np.allclose(y[:, 0], [w / 2, w / 8 + w])
    rng = np.random.default_rng(3)
    x, A, b = rng.normal(size=(1, 4, 1, 6)), rng.normal(size=1), rng.normal(size=(1, 6))
    # the decay gate with one rate a head, as a rate a channel
    assert np.allclose(gate(x, A, b)[0, :, 0], glr_gates(x[0, :, 0], np.repeat(A, 6), b[0])[1])


def test_recurrence_splits_anywhere():
    rng = np.random.default_rng(4)
    a = _glr_args(rng, 7, 3)
    y, final = glr(**a)
    for cut in range(8):
        first = dict(a, **{k: a[k][:cut] for k in ("x", "gate_x", "in_gate")})
        y1, s1 = glr(**first)
        y2, s2 = glr(**dict(a, **{k: a[k][cut:] for k in ("x", "gate_x", "in_gate")}, state=s1))
        assert np.allclose(np.concatenate([y1, y2]), y) and np.allclose(s2, final)


@pytest.mark.parametrize("T,in_gate,state,normalise", [(5, True, True, True), (4, False, True, False), (1, True, False, True),
                                                       (0, True, True, True)])
def test_recurrence_gradients(T, in_gate, state, normalise):
    rng = np.random.default_rng(5 + T)
    a = _glr_args(rng, T, 2, in_gate, state)
    dy, df = rng.normal(size=(T, 2)), rng.normal(size=2)

    def loss(**kw):
        y, f = glr(**dict(a, **kw), normalise=normalise)
        return float((y * dy).sum() + (f * df).sum())

    dx, dr, di, dA, db, dh = glr_bwd(a["x"], a["gate_x"], a["A_log"], dy, a["dt_bias"], a["in_gate"], a["state"], df, normalise)
    _differences(loss, a, dict(x=dx, gate_x=dr, in_gate=di if in_gate else None, A_log=dA, dt_bias=db,
                               state=dh if state else None))


def test_checkpoint_values():
    x = np.zeros((2, 64))
    x[0, 0], x[0, 1], x[0, 2], x[0, 3] = 448.0, 17.0, 2.0 ** -10, -3 * 2.0 ** -10
    x[0, 32] = 449.0
    x[1, 5], x[1, 6], x[1, 7], x[1, 8] = np.inf, np.nan, -np.inf, -1.0
    codes, byte = checkpoint_pack(x)
    assert byte.tolist() == [[127, 128], [119, 0]]  # 2^0, 2^1; 1 = 256 x 2^-8; nothing
    v = checkpoint_unpack(codes, byte)
    # ties to even: 17 between 16 and 18; 2^-10 between 0 and 2^-9; 3 2^-10 between 2^-9 and 2^-8
    assert v[0, :4].tolist() == [448.0, 16.0, 0.0, -2.0 ** -8] and v[0, 32] == 448.0
    assert np.isnan(v[1, 5:8]).all() and v[1, 8] == -1.0 and not v[1, 9:].any()
    again = checkpoint_pack(np.nan_to_num(v))
    assert np.array_equal(checkpoint_unpack(*again), np.nan_to_num(v))  # values of a checkpoint stay


def test_checkpoint_error():
    rng = np.random.default_rng(6)
    x = rng.normal(size=(50, 32)) * 10.0 ** rng.uniform(-6, 6, size=(50, 1))
    codes, byte = checkpoint_pack(x)
    scale = 2.0 ** (byte.astype(float) - 127)
    assert np.all(np.abs(x).max(-1, keepdims=True) <= 448 * scale) and np.all(np.abs(x).max(-1, keepdims=True) > 224 * scale)
    assert np.all(np.abs(checkpoint_unpack(codes, byte) - x) <= np.maximum(np.abs(x) * 2.0 ** -4, scale * 2.0 ** -10))
