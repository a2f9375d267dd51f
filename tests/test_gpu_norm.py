"""GPU parity of kda_prenorm_fwd / _bwd and kda_postnorm_fwd / _bwd against the float64 oracle.

Tolerance, per element, with u = 2^-24 and half a step of the output type on every stored value.
Forward: h carries e_h = 2u (|residual| + |scale x|) (product and addition; 0 for a plain x). A row's sum
of squares adds at most 32 terms a thread, 6 lane swaps and 16 waves, each within u, so its relative
error is under 64 u + 2 sum |h| e_h / sum h^2, and half of that reaches 1 / rms, with 6 u for division,
root and products: |err| <= |w| / rms e_h + |y| (that). A gate adds (8 + 2 |gate|) u (exp2 of a rounded
product, addition, reciprocal) relatively, scale and residual 2 u of their terms.
Backward: dv = T1 - T2, T1 = |u| / rms, T2 = |n| mean|u n| / rms taken in absolute values; each carries
the errors above on exact inputs, under (128 + 4 max|gate|) u of T1 + T2. The sums over rows add their
float32 terms in some order: (rows + 200 + 4 max|gate|) u of the absolute terms."""

import numpy as np
import pytest
import torch

import gated_delta_rule_67_amd as kda
from oracle import postnorm, postnorm_bwd, prenorm, prenorm_bwd
from tests.helpers import log, to64

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24
EPS = 1e-6


def close(got, ref, tol, what):
    got = to64(got)
    assert got.shape == ref.shape and np.all(np.isfinite(got)), what
    ratio = float(np.max(np.abs(got - ref) / (tol + 1e-300))) if ref.size else 0.0
    log(f"    {what}: worst |err| / tolerance {ratio:.3f}")
    assert ratio <= 1.0, f"{what}: {ratio}"


def _tensor(g, shape, dtype, pad):
    """A tensor of this shape; with pad, the last columns of a wider activation."""
    if not pad:
        return torch.randn(shape, generator=g).to(dtype).cuda()
    lead, width = (shape[:-2], shape[-2] * shape[-1]) if len(shape) > 2 else (shape[:-1], shape[-1])
    t = torch.randn(lead + (width + pad,), generator=g).to(dtype).cuda()[..., pad:]
    return t.unflatten(-1, shape[-2:]) if len(shape) > 2 else t


def _absolute_mean(v):
    return np.mean(v, axis=-1, keepdims=True)


def _values(t):
    """float64 of a tensor, or of a checkpoint."""
    if isinstance(t, tuple):
        return to64(kda.kda_checkpoint_unpack(t[0], t[1], torch.float32))
    return None if t is None else to64(t)


def _check_fwd(d, h, pre, silu, dtype):
    half = HALF[dtype]
    x, w, r, s, g = h["x"], h["weight"], h["residual"], h["scale"], h["gate"]
    if pre:
        y, hh = kda.kda_prenorm_fwd(d["x"], d["weight"], d["residual"], d["scale"], eps=EPS)
        ref, href = prenorm(x, w, r, s, EPS)
        eh = 2 * U * (np.abs(x if s is None else s * x) + (0 if r is None else np.abs(r)))
        if r is None and s is None:
            assert hh is d["x"]
            eh = 0 * eh
        else:
            close(hh, href, half * np.abs(href) + eh, "h")
        inv = 1 / np.sqrt(_absolute_mean(href ** 2) + EPS)
        rel = 0.5 * (64 * U + 2 * _absolute_mean(np.abs(href) * eh) / (_absolute_mean(href ** 2) + EPS)) + 6 * U
        close(y, ref, half * np.abs(ref) + np.abs(w) * inv * eh + np.abs(ref) * rel, "y")
        return hh
    y = kda.kda_postnorm_fwd(d["x"], d["weight"], d["gate"], d["residual"], d["scale"],
                             activation="silu" if silu else "sigmoid", eps=EPS)
    ref = postnorm(x, w, g, r, s, silu, EPS)
    part = ref if r is None else ref - r
    rel = (40 + (0 if g is None else 8 + 2 * np.abs(g))) * U
    close(y, ref, half * np.abs(ref) + np.abs(part) * rel + 2 * U * (np.abs(part) + (0 if r is None else np.abs(r))), "y")


def _check_bwd(d, h, pre, silu, dtype, rows):
    half = HALF[dtype]
    w, s, g, dy = h["weight"], h["scale"], h["gate"], h["dy"]
    inv_of = lambda v: 1 / np.sqrt(_absolute_mean(v ** 2) + EPS)  # noqa: E731
    total = lambda v: v.reshape(-1, v.shape[-1]).sum(0)  # noqa: E731
    if pre:
        got = kda.kda_prenorm_bwd(d["h"], d["weight"], d["dy"], d["dh"], d["x"], d["scale"], eps=EPS)
        v, x = h["h"], h["x"]
        ref = prenorm_bwd(v, w, dy, h["dh"], x, s, EPS)
        inner, k = w * dy, 0.0
    else:
        got = kda.kda_postnorm_bwd(d["x"], d["weight"], d["dy"], d["gate"], d["scale"],
                                   activation="silu" if silu else "sigmoid", eps=EPS)
        v = h["x"]
        ref = postnorm_bwd(v, w, dy, g, s, silu, EPS)
        act = 1.0 if g is None else np.abs(g if silu else 1.0) / (1 + np.exp(-g))
        inner = np.abs(dy * w * act * (1 if s is None else s))
        k = 0.0 if g is None else np.abs(g).max()
    inv = inv_of(v)
    n = np.abs(v * inv)
    T = inv * (np.abs(inner) + n * _absolute_mean(np.abs(inner) * n))
    e = (128 + 4 * k) * U
    es = (rows + 200 + 4 * k) * U
    tol = e * T
    if pre:
        tol = tol + (0 if h["dh"] is None else 2 * U * (np.abs(h["dh"]) + T))
        close(got[0], ref[0], half * np.abs(ref[0]) + tol, "dresidual")
        close(got[2], ref[2], es * total(np.abs(dy) * n) + U * np.abs(ref[2]), "dweight")
        if s is None:
            assert got[1] is got[0] and got[3] is None
        else:
            close(got[1], ref[1], half * np.abs(ref[1]) + np.abs(s) * (tol + 2 * U * np.abs(ref[0])), "dx")
            close(got[3], ref[3], total(np.abs(x) * (tol + es * (T + (0 if h["dh"] is None else np.abs(h["dh"]))))), "dscale")
        return
    close(got[0], ref[0], half * np.abs(ref[0]) + tol, "dx")
    d_abs = np.abs(dy * (1 if s is None else s))
    close(got[2], ref[2], es * total(d_abs * n * act), "dweight")
    if g is not None:
        sg = 1 / (1 + np.exp(-g))
        slope = sg * (1 + np.abs(g)) if silu else sg / (1 + np.exp(g))
        # silu's slope s (1 + z (1 - s)) in absolute terms: s (1 + |z|)
        close(got[1], ref[1], half * np.abs(ref[1]) + e * d_abs * np.abs(w) * n * slope, "dgate")
    else:
        assert got[1] is None
    if s is not None:
        close(got[3], ref[3], es * total(np.abs(dy * w) * n * act), "dscale")
    else:
        assert got[3] is None


def _run(shape, dtype, pre, residual=True, scale=True, gate=True, silu=False, pad=0, packed=False, seed=0):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    log(f"norm {shape} {dtype} pre={pre} residual={residual} scale={scale} gate={gate} silu={silu} pad={pad} packed={packed}")
    g = torch.Generator().manual_seed(seed + shape[-1])
    D = shape[-1]
    d = dict(weight=torch.randn(D, generator=g).cuda(), scale=torch.randn(D, generator=g).cuda() if scale else None,
             residual=_tensor(g, shape, dt, pad) if residual else None,
             gate=2 * _tensor(g, shape, dt, pad) if gate and not pre else None, x=_tensor(g, shape, dt, pad),
             dy=_tensor(g, shape, dt, pad), dh=_tensor(g, shape, dt, pad) if residual else None)
    h = {k: _values(v) for k, v in d.items()}
    hh = _check_fwd(d, h, pre, silu, dt)
    d["h"] = hh
    if packed:
        for k in ("x", "h", "gate"):
            if d[k] is not None:
                d[k] = kda.kda_checkpoint_pack(d[k])
    h.update({k: _values(d[k]) for k in ("x", "h", "gate")})
    _check_bwd(d, h, pre, silu, dt, int(np.prod(shape[:-1])))


WIDTHS = [1, 2, 7, 32, 64, 65, 128, 256, 520, 1030, 2048, 2052, 4095, 4100, 8191, 8192]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pre", [True, False])
def test_widths(D, dtype, pre):
    _run((5, D), dtype, pre)
    _run((1, D), dtype, pre, residual=False, scale=False, silu=True)


@pytest.mark.parametrize("residual,scale,gate,silu", [(False, False, False, False), (True, False, True, True),
                                                      (False, True, True, True), (True, True, False, False)])
@pytest.mark.parametrize("pre", [True, False])
def test_parts(residual, scale, gate, silu, pre):
    _run((3, 67, 128), "bf16", pre, residual, scale, gate, silu)
    _run((201, 130), "f32", pre, residual, scale, gate, silu)


@pytest.mark.parametrize("shape,pad", [((9, 4, 128), 8), ((2, 11, 3, 64), 64), ((2, 7, 136), 1), ((5, 2, 33), 3), ((40, 2048), 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pre", [True, False])
def test_slices_of_a_wider_activation(shape, pad, dtype, pre):
    _run(shape, dtype, pre, pad=pad)


@pytest.mark.parametrize("shape,pad", [((70, 32), 0), ((9, 4, 128), 0), ((33, 2048), 0), ((3, 8192), 0), ((3, 4128), 0),
                                       ((21, 96), 5), ((6, 2, 64), 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pre", [True, False])
def test_backward_from_checkpoints(shape, pad, dtype, pre):
    _run(shape, dtype, pre, pad=pad, packed=True)
    _run(shape, dtype, pre, residual=False, scale=False, gate=True, silu=True, packed=True)


@pytest.mark.parametrize("shape", [(300_001, 64), (6001, 1024)])
@pytest.mark.parametrize("pre", [True, False])
def test_more_rows_than_a_launch_holds_at_once(shape, pre):
    _run(shape, "bf16", pre)


def test_no_rows():
    w, s = torch.randn(48, device="cuda"), torch.randn(48, device="cuda")
    x = torch.empty((0, 48), device="cuda", dtype=torch.bfloat16)
    y, h = kda.kda_prenorm_fwd(x, w, x, s)
    assert y.shape == h.shape == (0, 48) and kda.kda_postnorm_fwd(x, w, x).shape == (0, 48)
    for out in (kda.kda_prenorm_bwd(h, w, y, None, x, s), kda.kda_postnorm_bwd(x, w, y, x, s)):
        assert out[0].shape == out[1].shape == (0, 48) and not out[2].any() and not out[3].any()


def test_rows_of_zeros_and_large_rows():
    """A row of zeros gives zeros (and a finite gradient); rows up to 2^60 and down to 2^-60 keep their norm."""
    w = torch.ones(96, device="cuda")
    x = torch.randn(4, 96, device="cuda")
    x[1] = 0
    x[2] *= 2.0 ** 55
    x[3] *= 2.0 ** -60
    y = kda.kda_postnorm_fwd(x, w, eps=1e-37)
    dx = kda.kda_postnorm_bwd(x, w, torch.ones_like(x), eps=1e-37)[0]
    assert not y[1].any() and bool(torch.isfinite(dx).all())
    close(y[2:], postnorm(to64(x[2:]), np.ones(96), eps=1e-37), 64 * U * np.abs(to64(y[2:])), "y")


@pytest.mark.parametrize("D", [64, 2048])
def test_rows_do_not_leak(D):
    """NaN and infinities in one row leave the others' outputs as they are."""
    torch.manual_seed(1)
    w, s = torch.randn(D, device="cuda"), torch.randn(D, device="cuda")
    x, r, z = (torch.randn(11, D, device="cuda").to(torch.bfloat16) for _ in range(3))
    bad = [t.clone() for t in (x, r, z)]
    bad[0][4, 3], bad[1][5, 0], bad[2][4, 1] = float("nan"), float("inf"), float("-inf")
    keep = [i for i in range(11) if i not in (4, 5)]
    for f in (lambda x, r, z: kda.kda_prenorm_fwd(x, w, r, s), lambda x, r, z: [kda.kda_postnorm_fwd(x, w, z, r, s)],
              lambda x, r, z: kda.kda_prenorm_bwd(x, w, r, z, x, s)[:2], lambda x, r, z: kda.kda_postnorm_bwd(x, w, r, z, s)[:2]):
        for a, b in zip(f(x, r, z), f(*bad)):
            assert torch.equal(a[keep], b[keep])


def test_large_offsets():
    """Tokens far enough apart that element offsets pass 32 bits."""
    T, D, ld = 9, 64, 300_000_000
    x = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").as_strided((T, D), (ld, 1))
    x.copy_(torch.randn(T, D))
    w, c = torch.randn(D, device="cuda"), x.contiguous()
    for f in (lambda t: kda.kda_prenorm_fwd(t, w, t)[0], lambda t: kda.kda_postnorm_fwd(t, w, t),
              lambda t: kda.kda_prenorm_bwd(t, w, t, t)[0], lambda t: kda.kda_postnorm_bwd(t, w, t, t)[1],
              lambda t: kda.kda_checkpoint_pack(t)[0].view(torch.uint8)):
        assert torch.equal(f(x), f(c))


def test_outputs_in_the_residuals_memory():
    lib = kda.library()
    T, D = 37, 520
    x, r = (torch.randn(T, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.randn(D, device="cuda")
    y, h = kda.kda_prenorm_fwd(x, w, r)
    z = kda.kda_postnorm_fwd(x, w, None, r)
    s = torch.cuda.current_stream().cuda_stream
    r1, r2, y1 = r.clone(), r.clone(), torch.empty_like(y)
    assert lib.kda_prenorm_fwd(x.data_ptr(), D, r1.data_ptr(), D, w.data_ptr(), None, y1.data_ptr(), r1.data_ptr(), T, 1, D,
                               1e-6, 1, s) == kda.KDA_OK
    assert lib.kda_postnorm_fwd(x.data_ptr(), D, w.data_ptr(), None, 0, r2.data_ptr(), D, None, r2.data_ptr(), T, 1, D, 1e-6,
                                0, 1, s) == kda.KDA_OK
    assert torch.equal(y1, y) and torch.equal(r1, h) and torch.equal(r2, z)


def test_repeats_bit_for_bit_on_a_side_stream_and_in_a_graph():
    torch.manual_seed(2)
    w, s = torch.randn(128, device="cuda"), torch.randn(128, device="cuda")
    x, r, z, dy = (torch.randn(3000, 4, 128, device="cuda").to(torch.bfloat16) for _ in range(4))

    def run():
        y, h = kda.kda_prenorm_fwd(x, w, r, s)
        out = [y, h, kda.kda_postnorm_fwd(x, w, z, r, s)]
        out += kda.kda_prenorm_bwd(h, w, dy, r, x, s)
        return out + list(kda.kda_postnorm_bwd(x, w, dy, z, s))

    ref = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        for t in got:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        assert all(torch.equal(a, b) for a, b in zip(run(), ref))
