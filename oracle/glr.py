"""The gated linear recurrence with one state per channel in float64 numpy, token by token, and its
gradients.

The decay is the standard gate's (K3 README, roadmap row L5), per channel:
g = -exp(A_log) softplus(gate_x + dt_bias), a = exp(g); h_t = a_t h_{t-1} + w_t logistic(in_gate_t)
x_t with w = sqrt(1 - a^2) or 1. One sequence [T, D] a call. Test infrastructure only.
"""

import numpy as np


def _logistic(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def glr_gates(gate_x, A_log, dt_bias=None, in_gate=None, normalise=True):
    """(z, g, a, w, s): the softplus' input, log decay, decay, input weight, input gate."""
    z = gate_x if dt_bias is None else gate_x + dt_bias
    g = -np.exp(A_log) * np.logaddexp(0.0, z)
    w = np.sqrt(-np.expm1(2.0 * g)) if normalise else np.ones_like(g)
    return z, g, np.exp(g), w, np.ones_like(g) if in_gate is None else _logistic(in_gate)


def glr(x, gate_x, A_log, dt_bias=None, in_gate=None, state=None, normalise=True):
    """(y, final state)."""
    _, _, a, w, s = glr_gates(gate_x, A_log, dt_bias, in_gate, normalise)
    h = np.zeros(x.shape[1]) if state is None else np.array(state, dtype=np.float64)
    y = np.zeros(x.shape)
    for t in range(len(x)):
        h = a[t] * h + w[t] * s[t] * x[t]
        y[t] = h
    return y, h


def glr_bwd(x, gate_x, A_log, dy, dt_bias=None, in_gate=None, state=None, dfinal=None, normalise=True):
    """(dx, dgate_x, din_gate, dA_log, ddt_bias, dstate) of <y, dy> + <final state, dfinal>."""
    z, g, a, w, s = glr_gates(gate_x, A_log, dt_bias, in_gate, normalise)
    y, _ = glr(x, gate_x, A_log, dt_bias, in_gate, state, normalise)
    before = np.concatenate([np.zeros((1, x.shape[1])) if state is None else np.asarray(state)[None], y[:-1]])[:len(x)]
    R = np.zeros(x.shape[1]) if dfinal is None else np.array(dfinal, dtype=np.float64)
    grad = np.zeros(x.shape)
    for t in reversed(range(len(x))):
        grad[t] = dy[t] + R
        R = a[t] * grad[t]
    dg = grad * a * before
    if normalise:
        dg = dg - grad * s * x * np.divide(a * a, w, out=np.zeros_like(w), where=w > 0)
    dz = -np.exp(A_log) * _logistic(z) * dg
    return (grad * s * w, dz, grad * x * w * s * (1.0 - s), (dg * g).sum(0), dz.sum(0), R)
