"""The norms around a block in float64 numpy, and their gradients.

In front (DM-KDAGQA-1.7B-SD model card, Model table: RMSNorm): h = residual + scale x,
y = weight h / sqrt(mean(h^2) + eps). Behind: y = residual + scale weight act(gate) x /
sqrt(mean(x^2) + eps), act the logistic or silu. Rows are the last axis. Test infrastructure only.
"""

import numpy as np


def _act(gate, silu):
    """act(gate) and its derivative."""
    if gate is None:
        return 1.0, None
    s, rest = 1.0 / (1.0 + np.exp(-gate)), 1.0 / (1.0 + np.exp(gate))
    return (gate * s, s * (1.0 + gate * rest)) if silu else (s, s * rest)


def _inv(v, eps):
    return 1.0 / np.sqrt(np.mean(v * v, axis=-1, keepdims=True) + eps)


def prenorm(x, weight, residual=None, scale=None, eps=1e-6):
    """(y, h)."""
    h = x if scale is None else scale * x
    h = h if residual is None else residual + h
    return weight * h * _inv(h, eps), h


def postnorm(x, weight, gate=None, residual=None, scale=None, silu=False, eps=1e-6):
    y = weight * _act(gate, silu)[0] * x * _inv(x, eps)
    y = y if scale is None else scale * y
    return y if residual is None else residual + y


def _back(v, u, eps):
    """Gradient of v for the gradient u of n = v inv, entry by entry of the Jacobian
    dn_i/dv_j = inv (delta_ij - n_i n_j / D)."""
    inv = _inv(v, eps)
    n = v * inv
    return inv * u - inv * n * np.sum(u * n, axis=-1, keepdims=True) / v.shape[-1]


def _rows(v):
    return v.reshape(-1, v.shape[-1]).sum(0)


def prenorm_bwd(h, weight, dy, dh=None, x=None, scale=None, eps=1e-6):
    """(dresidual, dx, dweight, dscale)."""
    d = _back(h, weight * dy, eps)
    d = d if dh is None else d + dh
    dweight = _rows(dy * h * _inv(h, eps))
    return (d, d, dweight, None) if scale is None else (d, scale * d, dweight, _rows(x * d))


def postnorm_bwd(x, weight, dy, gate=None, scale=None, silu=False, eps=1e-6):
    """(dx, dgate, dweight, dscale)."""
    act, slope = _act(gate, silu)
    d = dy if scale is None else scale * dy
    n = x * _inv(x, eps)
    return (_back(x, d * weight * act, eps), None if gate is None else d * weight * n * slope,
            _rows(d * n * act), None if scale is None else _rows(dy * weight * n * act))
