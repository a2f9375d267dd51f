"""GPU parity of kda_conv_fwd / kda_conv_bwd / kda_conv_step against the float64 oracle.

Tolerance, per element: half a step of the output type on the value, plus float32 rounding of
the sum: with A = |bias| + sum |weight| |x|, pre carries at most (W + 1) 2^-24 A. y = pre s(pre)
has slope at most 1.1 and its logistic a relative error under (8 + 2 |pre|) 2^-24 (hardware exp2 of
a rounded product, add, reciprocal), so |err| <= half step |y| + 2^-24 (1.1 (W + 1) A +
(8 + 2 |pre|) |pre|); with |pre| <= A: 2^-24 (16 + 2 A) A. Gradients: dpre = dy s' has |s'| <= 1.1
and slope at most 0.5, so its error is under 2^-24 (16 + 2 A) A |dy|, and every term of dx carries
it once; the sums over n tokens add n 2^-24 of their absolute terms (any order)."""

import numpy as np
import pytest
import torch

import gated_delta_rule_67_amd as kda
from oracle import conv, conv_bwd
from tests.helpers import log, to64

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F32 = 2.0 ** -24


def _make(lengths, D, W, dtype, seed, init=True, bias=True, tail=0, pad=0):
    g = torch.Generator().manual_seed(seed)
    T = sum(lengths) + tail
    wide = torch.randn((T, D + pad), generator=g).to(dtype)
    N = len(lengths)
    d = dict(x=wide, dy=torch.randn((T, D + pad), generator=g).to(dtype),
             weight=torch.randn((D, W), generator=g), bias=torch.randn(D, generator=g) if bias else None,
             init=torch.randn((N, W - 1, D), generator=g).to(dtype) if init else None,
             dfinal=torch.randn((N, W - 1, D), generator=g).to(dtype) if init else None,
             cu=torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32))
    d = {k: None if v is None else v.cuda() for k, v in d.items()}
    d["x"], d["dy"] = d["x"][:, pad:], d["dy"][:, pad:]
    return d


def _close(got, ref, tol, what):
    got = to64(got)
    assert got.shape == ref.shape and np.all(np.isfinite(got)), what
    ratio = float(np.max(np.abs(got - ref) / tol)) if ref.size else 0.0
    log(f"    {what}: worst |err| / tolerance {ratio:.3f}")
    assert ratio <= 1.0, f"{what}: {ratio}"


def _absolute(x, w, b, s):
    """A of every token, and of x rows in order (state ; tokens)."""
    rows = np.abs(np.concatenate([s, x]))
    A = np.zeros_like(x) + (0 if b is None else np.abs(b))
    for k in range(w.shape[1]):
        A = A + np.abs(w[:, k]) * rows[k:k + len(x)]
    return A


CASES = [
    # lengths, D, W, dtype, silu, init, bias, pad (columns in front of x's slice)
    ([1], 8, 4, "bf16", True, True, True, 0),
    ([0, 1, 2, 3, 4, 5, 0, 37], 64, 4, "bf16", True, True, True, 0),
    ([257], 520, 4, "bf16", True, False, True, 8),
    ([5, 300, 1, 0, 90], 1030, 3, "f32", True, True, True, 0),
    ([130, 3, 70], 33, 2, "bf16", False, True, False, 0),
    ([64, 64], 12, 3, "bf16", True, True, True, 5),
    ([700], 6, 4, "f32", False, True, True, 2),
    ([2] * 70 + [1] * 70, 24, 4, "f32", True, True, True, 0),
]


@pytest.mark.parametrize("lengths,D,W,dtype,silu,init,bias,pad", CASES)
@pytest.mark.parametrize("tail", [0, 9])
def test_packed(lengths, D, W, dtype, silu, init, bias, pad, tail):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    log(f"conv lengths={lengths[:8]} D={D} W={W} {dtype} silu={silu} tail={tail}")
    d = _make(lengths, D, W, dt, seed=sum(lengths) + D, init=init, bias=bias, tail=tail, pad=pad)
    y, final = kda.kda_conv_fwd(d["x"], d["weight"], d["bias"], d["init"], d["cu"], silu=silu)
    dx, dw, db, di = kda.kda_conv_bwd(d["x"], d["weight"], d["dy"], d["bias"], d["init"], d["dfinal"],
                                      d["cu"], silu=silu)
    torch.cuda.synchronize()
    h = {k: None if v is None else to64(v) for k, v in d.items()}
    rw, rb, aw, ab, ew, eb = 0, 0, 0, 0, 0, 0
    at = 0
    for n, L in enumerate(lengths):
        x, dy = h["x"][at:at + L], h["dy"][at:at + L]
        s = np.zeros((W - 1, D)) if h["init"] is None else h["init"][n]
        df = None if h["dfinal"] is None else h["dfinal"][n]
        A = _absolute(x, h["weight"], h["bias"], s)
        ry, rf = conv(x, h["weight"], h["bias"], s, silu)
        _close(y[at:at + L], ry, HALF[dt] * np.abs(ry) + F32 * (16 + 2 * A) * A + 1e-30, f"y of {n}")
        assert np.array_equal(to64(final[n]), rf)
        (rdx, dwn, dbn, rdi), (awn, abn) = conv_bwd(x, h["weight"], dy, h["bias"], s, df, silu)
        rw, rb, aw, ab = rw + dwn, rb + dbn, aw + awn, ab + abn
        # error of dpre per token, spread over the rows its taps read
        e = F32 * (16 + 2 * A) * (A + 1) * np.abs(dy)
        rows = np.concatenate([s, x])
        spread = np.zeros_like(rows)
        for k in range(W):
            spread[k:k + L] += np.abs(h["weight"][:, k]) * (e + 1.1 * (W + 1) * F32 * np.abs(dy))
            ew = ew + (e * np.abs(rows[k:k + L])).sum(0)
        if df is not None:
            spread[L:] += 2 * F32 * np.abs(df)
        eb = eb + e.sum(0)
        _close(dx[at:at + L], rdx, HALF[dt] * np.abs(rdx) + spread[W - 1:] + 1e-30, f"dx of {n}")
        if init:
            _close(di[n], rdi, HALF[dt] * np.abs(rdi) + spread[:W - 1] + 1e-30, f"dinitial of {n}")
        at += L
    n = sum(lengths)
    _close(dw, rw, n * F32 * aw + ew[:, None] + 1e-30, "dweight")
    if bias:
        _close(db, rb, n * F32 * ab + eb + 1e-30, "dbias")
    assert not y[at:].any() and not dx[at:].any()  # rows in no sequence


@pytest.mark.parametrize("B,T,D,W", [(3, 65, 40, 4), (4, 1, 16, 3), (1, 513, 24, 2)])
def test_dense_equals_packed(B, T, D, W):
    d = _make([T] * B, D, W, torch.bfloat16, seed=B + T, pad=8)
    a = kda.kda_conv_fwd(d["x"], d["weight"], d["bias"], d["init"], d["cu"])
    b = kda.kda_conv_fwd(d["x"].unflatten(0, (B, T)), d["weight"], d["bias"], d["init"])
    assert torch.equal(a[0], b[0].flatten(0, 1)) and torch.equal(a[1], b[1])
    a = kda.kda_conv_bwd(d["x"], d["weight"], d["dy"], d["bias"], d["init"], d["dfinal"], d["cu"])
    b = kda.kda_conv_bwd(d["x"].unflatten(0, (B, T)), d["weight"], d["dy"].unflatten(0, (B, T)),
                         d["bias"], d["init"], d["dfinal"])
    assert torch.equal(a[0], b[0].flatten(0, 1)) and all(torch.equal(u, v) for u, v in zip(a[1:], b[1:]))


@pytest.mark.parametrize("D,W,dtype,pad", [(64, 4, "bf16", 0), (1030, 3, "f32", 2), (33, 2, "bf16", 1),
                                           (8, 4, "f32", 0)])
def test_steps_equal_the_forward(D, W, dtype, pad):
    """Token by token on slots: bit for bit the forward's outputs and final state (the same
    operations in the same order); other slots and padded requests stay as they were."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    B, T = 5, 7
    d = _make([T] * B, D, W, dt, seed=D, pad=pad)
    y, final = kda.kda_conv_fwd(d["x"], d["weight"], d["bias"], d["init"], d["cu"])
    slots = torch.tensor([6, 0, 3, 8, 1], dtype=torch.int32).cuda()
    pool = torch.full((9, W - 1, D), float("nan"), dtype=dt).cuda()
    pool[slots.long()] = d["init"]
    x = d["x"].unflatten(0, (B, T))
    for t in range(T):
        out = kda.kda_conv_step(x[:, t], d["weight"], pool, d["bias"], slots)
        assert torch.equal(out, y.unflatten(0, (B, T))[:, t])
    assert torch.equal(pool[slots.long()], final)
    assert bool(pool[[2, 4, 5, 7]].isnan().all())
    before = pool.clone()
    pad_slots = torch.tensor([-1, 9, 2 ** 31 - 1, -2 ** 31, 0], dtype=torch.int32).cuda()
    out = kda.kda_conv_step(x[:, 0], d["weight"], pool, d["bias"], pad_slots)
    assert not out[:4].any() and torch.equal(pool[1:].nan_to_num(7), before[1:].nan_to_num(7))
    one = d["init"].clone()  # without slots: request n on state n
    out = kda.kda_conv_step(x[:, 0], d["weight"], one, d["bias"])
    assert torch.equal(out, y.unflatten(0, (B, T))[:, 0])


def test_rows_of_other_sequences_do_not_leak():
    d = _make([20, 30, 25], 16, 4, torch.bfloat16, seed=3, init=False)
    base = kda.kda_conv_fwd(d["x"], d["weight"], d["bias"], None, d["cu"])
    gbase = kda.kda_conv_bwd(d["x"], d["weight"], d["dy"], d["bias"], None, None, d["cu"])
    x, dy = d["x"].clone(), d["dy"].clone()
    x[20:50] = float("nan")
    dy[20:50] = float("inf")
    y = kda.kda_conv_fwd(x, d["weight"], d["bias"], None, d["cu"])
    g = kda.kda_conv_bwd(x, d["weight"], dy, d["bias"], None, None, d["cu"])
    for a, b in ((y[0], base[0]), (g[0], gbase[0])):
        assert torch.equal(a[:20], b[:20]) and torch.equal(a[50:], b[50:])


def test_c_entry_leaves_rows_in_no_sequence():
    """Without KDA_ZERO_REST the rows in no sequence keep their bytes, in front and behind."""
    lib = kda.library()
    T, D, W = 40, 24, 4
    mark = 2.0 ** 40  # no output comes near it
    x = torch.randn(T, D, device="cuda").to(torch.bfloat16)
    w = torch.randn(D, W, device="cuda")
    cu = torch.tensor([3, 3, 21, 30], dtype=torch.int32, device="cuda")
    y = torch.full((T, D), mark, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert lib.kda_conv_fwd(x.data_ptr(), D, w.data_ptr(), None, None, cu.data_ptr(), 3, None, y.data_ptr(),
                            T, D, W, kda.KDA_CONV_SILU, 1, s) == kda.KDA_OK
    ws = torch.empty(lib.kda_conv_bwd_workspace_size(T, D, W, 1), dtype=torch.uint8, device="cuda")
    dx = torch.full((T, D), mark, dtype=torch.bfloat16, device="cuda")
    assert lib.kda_conv_bwd(x.data_ptr(), D, w.data_ptr(), None, None, cu.data_ptr(), 3, y.data_ptr(), D, None,
                            dx.data_ptr(), None, None, None, T, D, W, kda.KDA_CONV_SILU, 1, ws.data_ptr(),
                            ws.numel(), s) == kda.KDA_OK
    torch.cuda.synchronize()
    for out in (y, dx):
        assert bool((out[:3] == mark).all()) and bool((out[30:] == mark).all())
        assert not bool((out[3:30] == mark).any())


@pytest.mark.parametrize("cu", [[0, 50, 20, 99], [-7, 5, 5, 1000], [9, 2, -3, 40], [60, 70, 80, 90]])
def test_malformed_offsets_stay_in_bounds(cu):
    """Offsets out of order or out of range are clamped: some result, in bounds, and it ends."""
    d = _make([20, 10, 10], 16, 4, torch.float32, seed=4)
    off = torch.tensor(cu, dtype=torch.int32).cuda()
    y, f = kda.kda_conv_fwd(d["x"], d["weight"], d["bias"], d["init"], off)
    g = kda.kda_conv_bwd(d["x"], d["weight"], d["dy"], d["bias"], d["init"], d["dfinal"], off)
    torch.cuda.synchronize()
    assert y.shape == d["x"].shape and f.shape == d["init"].shape and g[0].shape == y.shape


def test_no_tokens():
    d = _make([0, 0], 16, 4, torch.bfloat16, seed=5)
    y, f = kda.kda_conv_fwd(d["x"], d["weight"], d["bias"], d["init"], d["cu"])
    assert y.shape == (0, 16) and torch.equal(f, d["init"])
    dx, dw, db, di = kda.kda_conv_bwd(d["x"], d["weight"], d["dy"], d["bias"], d["init"], d["dfinal"], d["cu"])
    assert not dw.any() and not db.any() and torch.equal(di, d["dfinal"])


def test_large_channel_offsets():
    """Rows far enough apart that element offsets pass 32 bits (a slice of a wide activation)."""
    T, D, W, ld = 9, 8, 4, 300_000_000
    buf = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((T, D), (ld, 1))
    x.copy_(torch.randn(T, D))
    w = torch.randn(D, W, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    y, _ = kda.kda_conv_fwd(x, w, None, None, cu)
    y2, _ = kda.kda_conv_fwd(x.contiguous(), w, None, None, cu)
    assert torch.equal(y, y2)
    dy = torch.randn(T, D, device="cuda").to(torch.bfloat16)
    a = kda.kda_conv_bwd(x, w, dy, cu_seqlens=cu)
    b = kda.kda_conv_bwd(x.contiguous(), w, dy, cu_seqlens=cu)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_repeats_bit_for_bit_on_a_side_stream_and_in_a_graph():
    d = _make([700, 33, 400], 136, 4, torch.bfloat16, seed=6)

    def both():
        y, f = kda.kda_conv_fwd(d["x"], d["weight"], d["bias"], d["init"], d["cu"])
        return (y, f) + kda.kda_conv_bwd(d["x"], d["weight"], d["dy"], d["bias"], d["init"], d["dfinal"], d["cu"])

    ref = [t.clone() for t in both()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for _ in range(3):
        for t in got:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        assert all(torch.equal(a, b) for a, b in zip(both(), ref))
