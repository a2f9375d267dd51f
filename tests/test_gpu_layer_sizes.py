"""The layer operators at sizes whose loops run more than once: row blocks of several batches of rows
with ends at every phase, many row blocks, several requests a lane, many segments.

Tolerances as in test_gpu_conv.py and test_gpu_ssm.py, where they are derived."""

import numpy as np
import pytest
import torch

import gated_delta_rule_67_amd as kda
from oracle import conv, conv_bwd
from tests.helpers import log, to64
from tests.test_gpu_conv import F32, HALF, _absolute, _close, _make
from tests.test_gpu_ssm import _check as _check_ssm
from tests.test_gpu_ssm import _fwd as _ssm_fwd
from tests.test_gpu_ssm import _make as _make_ssm

pytestmark = pytest.mark.gpu

DT = dict(bf16=torch.bfloat16, f32=torch.float32)


def _check_conv(d, lengths, dtype, W, silu, channels):
    """Forward and backward of these channels against the oracle."""
    y, final = kda.kda_conv_fwd(d["x"], d["weight"], d["bias"], d["init"], d["cu"], silu=silu)
    dx, dw, db, di = kda.kda_conv_bwd(d["x"], d["weight"], d["dy"], d["bias"], d["init"], d["dfinal"], d["cu"], silu=silu)
    torch.cuda.synchronize()
    dt, ch = DT[dtype], torch.tensor(channels, device="cuda")
    pick = lambda t: None if t is None else to64(t.index_select(t.dim() - 1, ch))  # noqa: E731
    h = {k: pick(d[k]) for k in ("x", "dy", "bias", "init", "dfinal")}
    w = to64(d["weight"].index_select(0, ch))
    y, final, dx, di = pick(y), pick(final), pick(dx), pick(di)
    rw, rb, aw, ab, ew, eb, at = 0, 0, 0, 0, 0, 0, 0
    for n, L in enumerate(lengths):
        x, dy = h["x"][at:at + L], h["dy"][at:at + L]
        s, df = h["init"][n], h["dfinal"][n]
        A = _absolute(x, w, h["bias"], s)
        ry, rf = conv(x, w, h["bias"], s, silu)
        _close(torch.from_numpy(y[at:at + L]), ry, HALF[dt] * np.abs(ry) + F32 * (16 + 2 * A) * A + 1e-30, f"y of {n}")
        assert np.array_equal(final[n], rf)
        (rdx, dwn, dbn, rdi), (awn, abn) = conv_bwd(x, w, dy, h["bias"], s, df, silu)
        rw, rb, aw, ab = rw + dwn, rb + dbn, aw + awn, ab + abn
        e = F32 * (16 + 2 * A) * (A + 1) * np.abs(dy)
        rows = np.concatenate([s, x])
        spread = np.zeros_like(rows)
        for k in range(W):
            spread[k:k + L] += np.abs(w[:, k]) * (e + 1.1 * (W + 1) * F32 * np.abs(dy))
            ew = ew + (e * np.abs(rows[k:k + L])).sum(0)
        spread[L:] += 2 * F32 * np.abs(df)
        eb = eb + e.sum(0)
        _close(torch.from_numpy(dx[at:at + L]), rdx, HALF[dt] * np.abs(rdx) + spread[W - 1:] + 1e-30, f"dx of {n}")
        _close(torch.from_numpy(di[n]), rdi, HALF[dt] * np.abs(rdi) + spread[:W - 1] + 1e-30, f"dinitial of {n}")
        at += L
    T = sum(lengths)
    _close(dw.index_select(0, ch), rw, T * F32 * aw + ew[:, None] + 1e-30, "dweight")
    _close(db.index_select(0, ch), rb, T * F32 * ab + eb + 1e-30, "dbias")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("D,pad", [(6144, 0), (2050, 2)])
def test_convolution_with_long_slices(dtype, W, D, pad):
    """10 rows a wave or more (forward; 70 backward), so its loops over batches of four rows go round
    several times; sequences end at every phase of a batch and of a wave's slice, some of them shorter
    than the window."""
    lengths = [1501, 1, 2, 3, 0] + [37 + i for i in range(16)] + [64, 128, 4, 5, 6, 7] + [1701, 9001]
    log(f"conv D={D} W={W} {dtype}")
    d = _make(lengths, D, W, DT[dtype], seed=D + W, pad=pad)
    _check_conv(d, lengths, dtype, W, W != 3, [0, 1, 7, 8, 515, D // 2, D - 2, D - 1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_convolution_with_many_row_blocks(dtype):
    """Few channels: more than 112 row blocks, so the sums over them are read in batches."""
    lengths = [700, 1, 1900, 900]
    d = _make(lengths, 8, 4, DT[dtype], seed=8)
    _check_conv(d, lengths, dtype, 4, True, list(range(8)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B", [256, 257, 258, 259])
def test_convolution_steps_of_many_requests(dtype, B):
    """Several requests a lane, the last lanes with fewer, some without a slot; x is a slice of a wider
    activation. Bit for bit the forward's token."""
    D, W, pad, slots = 6144, 4, 64, 320
    d = _make([1] * B, D, W, DT[dtype], seed=B, pad=pad)
    y, final = kda.kda_conv_fwd(d["x"], d["weight"], d["bias"], d["init"], d["cu"])
    order = torch.randperm(slots, generator=torch.Generator().manual_seed(B))[:B].to(torch.int32)
    lost = torch.tensor([0, 5, 6, 130, B - 2, B - 1])
    where = order.clone()
    where[lost] = torch.tensor([-1, slots, 2 ** 31 - 1, -2 ** 31, -7, slots + 3], dtype=torch.int32)
    pool = torch.full((slots, W - 1, D), float("nan"), dtype=DT[dtype]).cuda()
    pool[order.long().cuda()] = d["init"]
    out = kda.kda_conv_step(d["x"], d["weight"], pool, d["bias"], where.cuda())
    keep = torch.ones(B, dtype=torch.bool)
    keep[lost] = False
    kept = keep.cuda()
    assert torch.equal(out[kept], y[kept]) and not out[~kept].any()
    assert torch.equal(pool[order.long().cuda()][kept], final[kept])
    assert torch.equal(pool[order.long().cuda()][~kept], d["init"][~kept])
    rest = torch.ones(slots, dtype=torch.bool)
    rest[order.long()] = False
    assert bool(pool[rest.cuda()].isnan().all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,tail", [([2900], 0), ([10, 2400, 0, 3, 700, 1, 1], 30)])
def test_scan_over_many_segments(dtype, lengths, tail):
    """More than eight boundaries in a row, so their composition goes round twice."""
    d, cu = _make_ssm(lengths, 2, 1, 64, 64, DT[dtype], seed=len(lengths), tail=tail)
    _check_ssm(d, cu, lengths, *_ssm_fwd(d, cu), dtype)


@pytest.mark.parametrize("B", [1, 3])
def test_scan_over_many_even_segments(B):
    T = 256 * 11
    d, cu = _make_ssm([T] * B, 2, 1, 64, 64, torch.bfloat16, seed=B)
    dense = {k: (v.unflatten(0, (B, T)) if k in ("x", "dt", "b", "c") else v) for k, v in d.items()}
    y, final = _ssm_fwd(dense, None)
    _check_ssm(d, cu, [T] * B, y.flatten(0, 1), final, "bf16")
