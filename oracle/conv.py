"""Short causal depthwise convolution in float64 numpy, token by token, and its gradients.

The layer in front of the KDA recurrence (KDA CUDA Trainer README, model paragraph; the
DM-KDAGQA-1.7B-SD model card's usage notes name its states): per channel,
pre_t = bias + sum_w weight[w] x_{t-(W-1)+w}, y = silu(pre) or pre, with W - 1 rows of state
in front of the first token. Test infrastructure only.
"""

import numpy as np


def _silu(pre):
    s = 1.0 / (1.0 + np.exp(-pre))
    return pre * s, s * (1.0 + pre * (1.0 - s))


def conv(x, weight, bias=None, state=None, silu=True):
    """One sequence: x [T, D], weight [D, W], bias [D], state [W-1, D]. Returns (y, final state)."""
    T, D = x.shape
    W = weight.shape[1]
    rows = np.concatenate([np.zeros((W - 1, D)) if state is None else state, x])
    y = np.zeros((T, D))
    for t in range(T):
        pre = np.zeros(D) if bias is None else np.array(bias, dtype=np.float64)
        for w in range(W):
            pre = pre + weight[:, w] * rows[t + w]
        y[t] = _silu(pre)[0] if silu else pre
    return y, rows[T:].copy()


def conv_bwd(x, weight, dy, bias=None, state=None, dfinal=None, silu=True):
    """Gradients of <y, dy> + <final state, dfinal> of one sequence:
    (dx, dweight, dbias, dstate), and the sums of |terms| of dweight and dbias."""
    T, D = x.shape
    W = weight.shape[1]
    rows = np.concatenate([np.zeros((W - 1, D)) if state is None else state, x])
    drows = np.zeros_like(rows)
    if dfinal is not None:
        drows[T:] += dfinal
    dweight, dbias = np.zeros((D, W)), np.zeros(D)
    aw, ab = np.zeros((D, W)), np.zeros(D)
    for t in range(T):
        pre = np.zeros(D) if bias is None else np.array(bias, dtype=np.float64)
        for w in range(W):
            pre = pre + weight[:, w] * rows[t + w]
        d = dy[t] * (_silu(pre)[1] if silu else 1.0)
        for w in range(W):
            drows[t + w] += weight[:, w] * d
            dweight[:, w] += d * rows[t + w]
            aw[:, w] += np.abs(d * rows[t + w])
        dbias += d
        ab += np.abs(d)
    return (drows[W - 1:], dweight, dbias, drows[:W - 1]), (aw, ab)
