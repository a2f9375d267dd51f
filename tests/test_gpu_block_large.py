"""The norms, the recurrence and the checkpoints on dense tensors of more than 2^31 (2^32) elements, on millions of
tiles and at the widest rows: equal, bit for bit, to calls on the last part alone, which the other tests compare
with the oracle.

A sequence's result depends on where its tiles and their groups lie on the tokens. Forward tiles have 120 tokens,
backward ones 64 (counted from the end), in groups of eight: parts that begin at a multiple of 8 x 1920 tokens have
the same ones."""

import pytest
import torch

import gated_delta_rule_67_amd as kda

pytestmark = pytest.mark.gpu


def _fill(t):
    """Random values in t, a piece at a time."""
    flat = t.view(-1)
    for first in range(0, flat.numel(), 1 << 27):
        part = flat[first:first + (1 << 27)]
        part.copy_(torch.randn(part.numel(), device="cuda", dtype=torch.float32))
    return t


def _equal(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_recurrence_over_many_tokens():
    """2^28 tokens: 2.2 million tiles forward, 4.2 million backward, over 2^31 elements."""
    torch.manual_seed(0)
    T, D, tail = (1 << 28) + 1920 * 8 * 7, 8, 1920 * 8 * 5
    x = _fill(torch.empty(T, D, dtype=torch.bfloat16, device="cuda"))
    A, b, init = torch.randn(D, device="cuda") - 4, torch.randn(D, device="cuda"), torch.randn(3, D, device="cuda")
    first = (T - tail) // (1920 * 8) * (1920 * 8)
    assert T % 64 == 0 and T * D > 1 << 31
    cu = torch.tensor([0, 1000, first, T], dtype=torch.int32, device="cuda")
    one = torch.tensor([0, T - first], dtype=torch.int32, device="cuda")
    y, f, s = kda.kda_glr_fwd(x, x, A, b, x, init, cu, output_block_states=True)
    y1, f1, s1 = kda.kda_glr_fwd(x[first:], x[first:], A, b, x[first:], init[2:], one, output_block_states=True)
    assert _equal(y[first:], y1) and torch.equal(f[2:], f1) and torch.equal(s[first // 64 + 1:], s1[1:])
    assert bool(torch.isfinite(y[first - 4096:first].float()).all())
    # the middle sequence against its last tokens from its state there: each side within 60 units of 2^-24 a token
    # (test_gpu_glr) of the largest state, and half a step of bf16
    mid = first - 960
    at = torch.tensor([0, first - mid], dtype=torch.int32, device="cuda")
    y2, f2 = kda.kda_glr_fwd(x[mid:first], x[mid:first], A, b, x[mid:first], s[mid // 64:mid // 64 + 1], at)
    scale = float(y2.float().abs().max())
    near = 2 * 960 * 60 * 2.0 ** -24 * scale
    assert float((y[mid:first].float() - y2.float()).abs().max()) <= near + 2.0 ** -7 * scale
    assert float((f[1:2] - f2).abs().max()) <= near
    del y, y1, y2
    g = kda.kda_glr_bwd(x, x, A, x, b, x, init, init, cu, block_states=s)
    g1 = kda.kda_glr_bwd(x[first:], x[first:], A, x[first:], b, x[first:], init[2:], init[2:], one, block_states=s1)
    for a, c in zip(g[:3], g1[:3]):
        assert _equal(a[first:], c) and bool(torch.isfinite(a[:4096].float()).all())
    assert torch.equal(g[5][2:], g1[5]) and bool(torch.isfinite(g[3]).all() and torch.isfinite(g[4]).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_recurrence_of_the_widest_rows(dtype):
    torch.manual_seed(1)
    T, D = 200, 1 << 20
    x = _fill(torch.empty(T, D, dtype=dtype, device="cuda"))
    A, b, init = torch.randn(D, device="cuda"), torch.randn(D, device="cuda"), torch.randn(2, D, device="cuda")
    cu = torch.tensor([0, 130, T], dtype=torch.int32, device="cuda")

    def run(c):
        v = x[:, c]
        args = (A[c].contiguous(), b[c].contiguous(), init[:, c].contiguous())
        out = kda.kda_glr_fwd(v, v, args[0], args[1], v, args[2], cu, output_block_states=True)
        return out + kda.kda_glr_bwd(v, v, args[0], v, args[1], v, args[2], args[2], cu, block_states=out[2])

    whole = run(slice(0, D))
    for c in (slice(0, 256), slice(D // 2, D // 2 + 256), slice(D - 256, D)):
        for i, (a, v) in enumerate(zip(whole, run(c))):
            # no state is kept where token 64 k begins a sequence: 0 here
            assert torch.equal(a[..., c], v) if i != 2 else torch.equal(a[1:, c], v[1:])
    pool = torch.randn(3, D, device="cuda")
    few = pool.clone()
    y = kda.kda_glr_step(x[:2], x[:2], A, pool, b, x[:2])
    c = slice(D - 100, D)
    small = few[:, c].contiguous()
    y1 = kda.kda_glr_step(x[:2, c], x[:2, c], A[c].contiguous(), small, b[c].contiguous(), x[:2, c])
    assert torch.equal(y[:, c], y1) and torch.equal(pool[:, c], small) and torch.equal(pool[2], few[2])


def test_norms_of_many_rows():
    torch.manual_seed(2)
    n, D = (1 << 21) + 3, 2048
    x = _fill(torch.empty(n, D, dtype=torch.bfloat16, device="cuda"))
    w, s = torch.randn(D, device="cuda"), torch.randn(D, device="cuda")
    last = slice(n - 5, n)
    for call in (lambda x: kda.kda_prenorm_fwd(x, w, x, s), lambda x: [kda.kda_postnorm_fwd(x, w, x, x, s)],
                 lambda x: kda.kda_prenorm_bwd(x, w, x, x, x, s)[:2], lambda x: kda.kda_postnorm_bwd(x, w, x, x, s)[:2]):
        for a, b in zip(call(x), call(x[last])):
            assert _equal(a[last], b)
        del a


def test_norms_of_narrow_rows():
    """2^30 rows of one column."""
    n = 1 << 30
    x = _fill(torch.empty(n, 1, dtype=torch.bfloat16, device="cuda"))
    w = torch.randn(1, device="cuda")
    y = kda.kda_postnorm_fwd(x, w)
    dx = kda.kda_postnorm_bwd(x, w, x)
    last = slice(n - 100, n)
    assert _equal(y[last], kda.kda_postnorm_fwd(x[last], w)) and _equal(dx[0][last], kda.kda_postnorm_bwd(x[last], w, x[last])[0])


def test_checkpoints_of_many_tokens():
    n, D = (1 << 26) + 5, 64
    x = _fill(torch.empty(n, D, dtype=torch.bfloat16, device="cuda"))
    codes, scales = kda.kda_checkpoint_pack(x)
    assert x.numel() > 1 << 32
    for c in (slice(n - 100, n), slice((1 << 25) - 50, (1 << 25) + 50)):
        part = kda.kda_checkpoint_pack(x[c])
        assert _equal(codes[c], part[0]) and torch.equal(scales[c], part[1])
    y = kda.kda_checkpoint_unpack(codes, scales)
    for c in (slice(n - 100, n), slice((1 << 25) - 50, (1 << 25) + 50)):
        assert _equal(y[c], kda.kda_checkpoint_unpack(codes[c], scales[c]))
