"""Pins of the selective scan oracle on the CPU: a hand-worked example, the explicit sum over
earlier tokens, the split at any token, and the KDA recurrence with beta = 0 prediction."""

import numpy as np

from oracle import selective_scan
from oracle.ssm import softplus


def _inputs(T=7, HV=4, H=2, K=3, V=2, seed=0):
    r = np.random.default_rng(seed)
    return dict(x=r.normal(size=(T, HV, V)), dt=r.normal(size=(T, HV)), A_log=r.normal(size=HV),
                b=r.normal(size=(T, H, K)), c=r.normal(size=(T, H, K)), D=r.normal(size=HV),
                dt_bias=r.normal(size=HV), state=r.normal(size=(HV, K, V)))


def test_hand_worked():
    # softplus(log(e - 1)) = 1, A_log = log(log 2): the state halves every token
    z = np.log(np.e - 1.0)
    y, S, _, _ = selective_scan(np.array([[[3.0]], [[5.0]]]), np.full((2, 1), z), np.array([np.log(np.log(2.0))]),
                                np.array([[[1.0]], [[2.0]]]), np.array([[[1.0]], [[-1.0]]]), np.array([10.0]),
                                None, np.array([[[4.0]]]))
    assert np.allclose(S, 0.5 * (0.5 * 4 + 3) + 10)
    assert np.allclose(y[:, 0, 0], [5 + 30, -12.5 + 50])


def test_against_the_explicit_sum():
    a = _inputs()
    y, S, ya, sa = selective_scan(**a)
    T, HV, V = a["x"].shape
    d = softplus(a["dt"] + a["dt_bias"])
    g = -np.exp(a["A_log"]) * d
    for h in range(HV):
        b, c = a["b"][:, h // 2], a["c"][:, h // 2]
        for t in range(T):
            out = a["D"][h] * a["x"][t, h] + np.exp(g[:t + 1, h].sum()) * (a["state"][h].T @ c[t])
            for s in range(t + 1):
                out = out + np.exp(g[s + 1:t + 1, h].sum()) * (b[s] @ c[t]) * d[s, h] * a["x"][s, h]
            assert np.allclose(y[t, h], out)
    assert np.all(ya >= np.abs(y) - 1e-12) and np.all(sa >= np.abs(S) - 1e-12)


def test_split_anywhere():
    a = _inputs(seed=1)
    y, S, _, _ = selective_scan(**a)
    for cut in range(8):
        first = {k: (v[:cut] if k in ("x", "dt", "b", "c") else v) for k, v in a.items()}
        y1, s1, _, _ = selective_scan(**first)
        rest = {k: (v[cut:] if k in ("x", "dt", "b", "c") else v) for k, v in a.items()}
        y2, s2, _, _ = selective_scan(**dict(rest, state=s1))
        assert np.allclose(np.concatenate([y1, y2]), y) and np.allclose(s2, S)
