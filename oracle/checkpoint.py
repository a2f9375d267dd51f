"""Activation checkpoints in 8 bits, from the table of e4m3 values: per 32 neighbours the smallest
power of two, 2^-127 at least, that brings the largest finite magnitude to 448 or less; codes by the
nearest table entry, ties to the even code; what is not finite becomes the NaN code.
Test infrastructure only."""

import numpy as np

# e4m3 without infinities: sign, 4 bits of exponent (bias 7), 3 of mantissa; 0x7f is NaN
MAGNITUDES = np.array([(c % 8) * 2.0 ** -9 if c < 8 else (1 + c % 8 / 8) * 2.0 ** (c // 8 - 7) for c in range(127)])


def checkpoint_pack(x):
    """x [..., D] -> (codes uint8 [..., D], scale bytes uint8 [..., D/32])."""
    x = np.asarray(x, dtype=np.float64)
    blocks = x.reshape(x.shape[:-1] + (-1, 32))
    top = np.max(np.where(np.isfinite(blocks), np.abs(blocks), 0.0), axis=-1)
    byte = np.zeros(top.shape, dtype=np.int64)
    for b in range(255):
        byte = np.where(top > 448.0 * 2.0 ** (b - 127), b + 1, byte)
    v = np.abs(blocks) / 2.0 ** (byte[..., None] - 127.0)
    v = np.where(np.isfinite(v), v, 0.0)
    up = np.clip(np.searchsorted(MAGNITUDES, v), 1, 126)
    lo, hi = v - MAGNITUDES[up - 1], MAGNITUDES[up] - v
    code = np.where((lo < hi) | ((lo == hi) & (up % 2 == 1)), up - 1, up)
    code = np.where(np.signbit(blocks), code + 128, code)
    code = np.where(np.isfinite(blocks), code, 127)
    return code.reshape(x.shape).astype(np.uint8), byte.astype(np.uint8)


def checkpoint_unpack(codes, byte):
    m = np.concatenate([MAGNITUDES, [np.nan]])
    table = np.concatenate([m, -m])
    return table[codes] * np.repeat(2.0 ** (byte.astype(np.float64) - 127.0), 32, axis=-1)
