"""Selective state space scan with a scalar decay per head, float64 numpy, token by token.

Per value head: D_t = softplus(dt_t + dt_bias), a_t = exp(-exp(A_log) D_t),
S_t = a_t S_{t-1} + b_t (D_t x_t)^T, y_t = S_t^T c_t + D x_t; value head hv reads b / c pair
hv // (HV // H). The decay is the KDA gate's standard form (K3 README, roadmap row L5). Test
infrastructure only.
"""

import numpy as np


def softplus(z):
    return np.maximum(z, 0.0) + np.log1p(np.exp(-np.abs(z)))


def selective_scan(x, dt, A_log, b, c, D=None, dt_bias=None, state=None):
    """One sequence: x [T,HV,V], dt [T,HV], A_log, D, dt_bias [HV], b, c [T,H,K], state [HV,K,V].
    Returns (y, final state, absolute y, absolute state): the last two are the sums of the
    absolute values of the terms of each element."""
    T, HV, V = x.shape
    H, K = b.shape[1:]
    G = HV // H
    S = np.zeros((HV, K, V)) if state is None else np.array(state, dtype=np.float64)
    A = np.abs(S)
    y, ya = np.zeros((T, HV, V)), np.zeros((T, HV, V))
    for t in range(T):
        d = softplus(dt[t] + (0.0 if dt_bias is None else dt_bias))
        a = np.exp(-np.exp(A_log) * d)
        bt, ct = np.repeat(b[t], G, axis=0), np.repeat(c[t], G, axis=0)
        S = a[:, None, None] * S + bt[:, :, None] * (d[:, None] * x[t])[:, None, :]
        A = a[:, None, None] * A + np.abs(bt[:, :, None] * (d[:, None] * x[t])[:, None, :])
        y[t] = (S * ct[:, :, None]).sum(1)
        ya[t] = (A * np.abs(ct)[:, :, None]).sum(1)
        if D is not None:
            y[t] += D[:, None] * x[t]
            ya[t] += np.abs(D[:, None] * x[t])
    return y, S, ya, A
