"""GPU parity of kda_ssm_chunk_fwd / kda_ssm_step against the float64 oracle.

Tolerance, per element, with A the sum of the absolute values of the element's terms (the oracle
gives it for y and for the state). float32 arithmetic: a sum of up to 128 + 64 products in any
order is within 192 2^-24 A < 2^-16 A, the softplus and the exponentials add under 2^-19 A (a
decay's relative error is 2^-20 of its exponent, and e^-u u < 1/2): 2^-15 A in all, for the state
of either type (bf16's update splits its weighted x into 24 bits) and for float32's y. bf16's y:
one rounding of every term (2^-8, of M or of S) and one of the result: 2^-8 (A + |y|) + 2^-15 A.
Over a whole tensor float32 errors do not add up one way: RMS(err) <= 2^-19 RMS(A)."""

import numpy as np
import pytest
import torch

import gated_delta_rule_67_amd as kda
from oracle import selective_scan
from tests.helpers import log, to64

pytestmark = pytest.mark.gpu

DT = dict(bf16=torch.bfloat16, f32=torch.float32)
TOKEN = ("x", "dt", "b", "c")


def _make(lengths, HV, H, K, V, dtype, seed, init=True, skip=True, bias=True, tail=0, pad=0, rate=1.0, strides=True):
    """Packed inputs on the GPU; x, b and c are slices of one activation (pad columns in front)."""
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lengths) + tail, len(lengths)
    act = torch.randn((T, pad + HV * V + 2 * H * K), generator=g).to(dtype).cuda()
    d = dict(x=act[:, pad:pad + HV * V].unflatten(1, (HV, V)),
             b=act[:, pad + HV * V:pad + HV * V + H * K].unflatten(1, (H, K)),
             c=act[:, pad + HV * V + H * K:].unflatten(1, (H, K)))
    if not strides:
        d = {k: v.contiguous() for k, v in d.items()}
    d.update(dt=(torch.randn((T, HV), generator=g) - 1.5).to(dtype).cuda(),
             A_log=torch.log(rate * (1 + 15 * torch.rand(HV, generator=g))).cuda(),
             D=torch.randn(HV, generator=g).cuda() if skip else None,
             dt_bias=(0.5 * torch.randn(HV, generator=g)).cuda() if bias else None,
             state=torch.randn((N, HV, K, V), generator=g).cuda() if init else None)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()
    return d, cu


def _fwd(d, cu, **kw):
    return kda.kda_ssm_chunk_fwd(d["x"], d["dt"], d["A_log"], d["b"], d["c"], d["D"], d["dt_bias"], d["state"], cu, **kw)


def _worst(got, ref, tol, what, rms_of=None):
    got = to64(got)
    assert got.shape == ref.shape and np.all(np.isfinite(got)), what
    if not ref.size:
        return
    err = np.abs(got - ref)
    ratio = float(np.max(err / tol))
    rms = float(np.sqrt(np.mean(err ** 2)) / np.sqrt(np.mean(rms_of ** 2))) if rms_of is not None else 0.0
    log(f"    {what}: worst |err| / tolerance {ratio:.3f}, rms err / rms A {rms:.2e}")
    assert ratio <= 1.0, f"{what}: {ratio}"
    assert rms <= 2.0 ** -19, f"{what}: rms {rms}"


def _check(d, cu, lengths, y, final, dtype, heads=None):
    h = {k: None if v is None else to64(v) for k, v in d.items()}
    HV, H = h["x"].shape[1], h["b"].shape[1]
    hs = list(range(HV)) if heads is None else heads
    at = 0
    for n, L in enumerate(lengths):
        one = dict(x=h["x"][at:at + L][:, hs], dt=h["dt"][at:at + L][:, hs], A_log=h["A_log"][hs],
                   b=h["b"][at:at + L][:, [i // (HV // H) for i in hs]], c=h["c"][at:at + L][:, [i // (HV // H) for i in hs]],
                   D=None if h["D"] is None else h["D"][hs], dt_bias=None if h["dt_bias"] is None else h["dt_bias"][hs],
                   state=None if h["state"] is None else h["state"][n][hs])
        ry, rs, ya, sa = selective_scan(**one)
        f32 = 2.0 ** -15
        if dtype == "f32":
            _worst(y[at:at + L][:, hs], ry, f32 * ya + 1e-30, f"y of {n} ({L})", ya)
        else:
            _worst(y[at:at + L][:, hs], ry, 2.0 ** -8 * (ya + np.abs(ry)) + f32 * ya + 1e-30, f"y of {n} ({L})")
        if final is not None:
            _worst(final[n][hs], rs, f32 * sa + 1e-30, f"state of {n}", sa if L else None)
            if L == 0:
                assert np.array_equal(to64(final[n][hs]), rs)
        at += L
    assert not y[at:].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("HV,H,K,V", [(2, 1, 128, 64), (4, 2, 64, 64), (1, 1, 128, 128), (3, 3, 128, 64),
                                      (4, 1, 32, 32), (3, 1, 40, 27), (2, 2, 33, 100), (1, 1, 1, 1), (2, 1, 16, 8), (2, 1, 24, 40),
                                      (1, 1, 56, 72), (2, 2, 8, 120)])
def test_shapes(dtype, HV, H, K, V):
    lengths = [1, 63, 64, 65, 0, 130]
    log(f"ssm {dtype} HV={HV} H={H} K={K} V={V}")
    d, cu = _make(lengths, HV, H, K, V, DT[dtype], seed=HV + K + V)
    _check(d, cu, lengths, *_fwd(d, cu), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,tail", [([1], 0), ([2, 2, 2, 2, 2, 2, 2, 2, 2], 5), ([700], 0), ([0, 0, 300, 0, 517, 0], 40),
                                          ([256, 256, 256, 255, 1], 0), ([1030, 3], 0), ([5] * 60, 0)])
def test_lengths(dtype, lengths, tail):
    """Several segments (256 tokens at least) with boundaries inside sequences, on their ends and
    in front of one-token sequences; rows behind the last sequence."""
    d, cu = _make(lengths, 2, 1, 64, 64, DT[dtype], seed=sum(lengths), tail=tail)
    _check(d, cu, lengths, *_fwd(d, cu), dtype)


@pytest.mark.parametrize("kw", [dict(init=False), dict(skip=False, bias=False), dict(pad=8), dict(pad=3),
                                dict(strides=False), dict(rate=200.0), dict(rate=1e-4), dict(rate=20.0)])
def test_options(kw):
    lengths = [400, 77]
    for dtype in ("bf16", "f32"):
        d, cu = _make(lengths, 4, 2, 64, 32, DT[dtype], seed=9, **kw)
        _check(d, cu, lengths, *_fwd(d, cu), dtype)
        y, none = _fwd(d, cu, output_final_state=False)
        assert none is None and torch.equal(y, _fwd(d, cu)[0])


def test_a_reset_then_slow_decay():
    """One token that all but clears the state, followed by tokens that hardly decay: differences
    of large sums of log decays keep their accuracy."""
    d, cu = _make([300], 2, 1, 64, 64, torch.float32, seed=2, rate=1.0)
    d["dt"] = torch.full_like(d["dt"], -6.0)
    d["dt"][100:130] = 80.0
    _check(d, cu, [300], *_fwd(d, cu), "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decays_past_every_float(dtype):
    """exp(A_log) overflows float32: the state holds the last token alone, and nothing is NaN."""
    d, cu = _make([70, 300], 2, 1, 64, 64, DT[dtype], seed=12)
    d["A_log"] = torch.tensor([100.0, 60.0]).cuda()
    _check(d, cu, [70, 300], *_fwd(d, cu), dtype)
    pool = d["state"].clone()
    y = kda.kda_ssm_step(d["x"][:2], d["dt"][:2], d["A_log"], d["b"][:2], d["c"][:2], pool, d["D"], d["dt_bias"])
    assert bool(y.isfinite().all()) and bool(pool.isfinite().all())


def test_rows_in_front_of_and_behind_the_sequences():
    """Whole segments of rows in no sequence, on both sides."""
    d, _ = _make([900], 2, 1, 64, 64, torch.bfloat16, seed=13, init=False)
    cu = torch.tensor([300, 300, 610], dtype=torch.int32).cuda()
    y, f = kda.kda_ssm_chunk_fwd(d["x"], d["dt"], d["A_log"], d["b"], d["c"], d["D"], d["dt_bias"], None, cu)
    one = {k: (v[300:610] if k in TOKEN else v) for k, v in d.items()}
    ry, rf = _fwd(one, torch.tensor([0, 310], dtype=torch.int32).cuda())
    assert not y[:300].any() and not y[610:].any() and not f[0].any()
    assert float((y[300:610].float() - ry.float()).abs().max()) <= 2.0 ** -6 * float(ry.float().abs().max())
    assert float((f[1] - rf[0]).abs().max()) <= 2.0 ** -15 * float(rf.abs().max())


def test_binding_refuses():
    d, cu = _make([64], 2, 1, 64, 64, torch.bfloat16, seed=14)
    ok = dict(x=d["x"], dt=d["dt"], A_log=d["A_log"], b=d["b"], c=d["c"], D=d["D"], dt_bias=d["dt_bias"],
              initial_state=d["state"], cu_seqlens=cu)
    kda.kda_ssm_chunk_fwd(**ok)
    for bad in (dict(x=d["x"].float()), dict(x=d["x"].transpose(0, 1)), dict(x=d["x"][:1].expand(64, 2, 64)),
                dict(dt=d["dt"][:-1]), dict(b=d["b"][..., :32]), dict(c=d["c"].cpu()), dict(A_log=d["A_log"].double()),
                dict(D=d["D"][:1]), dict(initial_state=d["state"].bfloat16()), dict(cu_seqlens=cu.long()),
                dict(cu_seqlens=cu[:1]), dict(cu_seqlens=None), dict(x=d["x"].half(), dt=d["dt"].half())):
        with pytest.raises(ValueError):
            kda.kda_ssm_chunk_fwd(**dict(ok, **bad))
    pool = d["state"].clone()
    for bad in (pool.bfloat16(), pool[:, :1], pool.transpose(2, 3)):
        with pytest.raises(ValueError):
            kda.kda_ssm_step(d["x"][:1], d["dt"][:1], d["A_log"], d["b"][:1], d["c"][:1], bad)
    with pytest.raises(ValueError):
        kda.kda_ssm_step(d["x"][:2], d["dt"][:2], d["A_log"], d["b"][:2], d["c"][:2], pool)  # one state, two requests
    w = torch.randn(8, 4).cuda()
    x = torch.randn(2, 6, 8).cuda()
    for call in (lambda: kda.kda_conv_fwd(x[:, 1:], w), lambda: kda.kda_conv_fwd(x, w.t()), lambda: kda.kda_conv_fwd(x, w.half()),
                 lambda: kda.kda_conv_fwd(x[..., ::2], w[::2]), lambda: kda.kda_conv_bwd(x, w, x[:1]),
                 lambda: kda.kda_conv_fwd(x, w, None, x[:, :2]), lambda: kda.kda_conv_step(x[:, 0], w, x[:, :2]),
                 lambda: kda.kda_slots_copy([x, x], cu[:1], cu[:1]), lambda: kda.kda_slots_copy([x, x[:1]], cu[:1], cu[:1]),
                 lambda: kda.kda_slots_copy(x.transpose(0, 1), cu[:1], cu[:1]), lambda: kda.kda_slots_copy(x, cu[:1], cu),
                 lambda: kda.kda_slots_compact(x, cu)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(RuntimeError):
        kda.kda_conv_fwd(x, torch.randn(8, 5).cuda())  # no kernel of this width


@pytest.mark.parametrize("B,T", [(3, 64), (2, 321), (4, 1), (1, 2048), (2, 1024)])
def test_dense_batches(B, T):
    for dtype in ("bf16", "f32"):
        d, cu = _make([T] * B, 4, 2, 64, 64, DT[dtype], seed=B * T)
        dense = {k: (v.unflatten(0, (B, T)) if k in TOKEN else v) for k, v in d.items()}
        y, final = _fwd(dense, None)
        assert y.shape == (B, T, 4, 64)
        _check(d, cu, [T] * B, y.flatten(0, 1), final, dtype, heads=[0, 3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("HV,H,K,V", [(4, 2, 128, 64), (2, 1, 64, 128), (3, 1, 33, 27), (1, 1, 1, 1), (16, 1, 128, 16)])
def test_steps(dtype, HV, H, K, V):
    """Steps on scattered slots against the oracle; the other slots keep their bytes, requests
    without a slot give zeros."""
    B, T = 5, 6
    d, cu = _make([T] * B, HV, H, K, V, DT[dtype], seed=K + V, pad=0)
    slots = torch.tensor([6, 0, 3, 8, 1], dtype=torch.int32).cuda()
    pool = torch.full((9, HV, K, V), float("nan")).cuda()
    pool[slots.long()] = d["state"]
    tok = {k: d[k].unflatten(0, (B, T)) for k in TOKEN}
    ys = [kda.kda_ssm_step(tok["x"][:, t], tok["dt"][:, t], d["A_log"], tok["b"][:, t], tok["c"][:, t], pool, d["D"],
                           d["dt_bias"], slots) for t in range(T)]
    y = torch.stack(ys, 1).flatten(0, 1)
    _check(d, cu, [T] * B, y, pool[slots.long()], dtype)
    assert bool(pool[[2, 4, 5, 7]].isnan().all())
    before = pool.clone()
    none = torch.tensor([-1, 9, 2 ** 31 - 1, -2 ** 31, 7], dtype=torch.int32).cuda()
    one = kda.kda_ssm_step(tok["x"][:, 0], tok["dt"][:, 0], d["A_log"], tok["b"][:, 0], tok["c"][:, 0], pool, d["D"], d["dt_bias"], none)
    keep = [0, 1, 2, 3, 4, 5, 6, 8]
    assert not one[:4].any() and torch.equal(pool[keep].nan_to_num(7), before[keep].nan_to_num(7))
    own = d["state"].clone()  # without slots: request n on state n
    one = kda.kda_ssm_step(tok["x"][:, 0], tok["dt"][:, 0], d["A_log"], tok["b"][:, 0], tok["c"][:, 0], own, d["D"], d["dt_bias"])
    assert torch.equal(one, ys[0])


def test_many_requests_one_step():
    d, cu = _make([1] * 300, 8, 2, 32, 64, torch.bfloat16, seed=4)
    pool = d["state"].clone()
    y = kda.kda_ssm_step(d["x"], d["dt"], d["A_log"], d["b"], d["c"], pool, d["D"], d["dt_bias"])
    _check(d, cu, [1] * 300, y, pool, "bf16", heads=[0, 7])


def test_rows_of_other_sequences_do_not_leak():
    d, cu = _make([100, 90, 400], 2, 1, 64, 64, torch.bfloat16, seed=3)
    y0, s0 = _fwd(d, cu)
    for k in ("x", "b", "c", "dt"):
        v = d[k].contiguous().clone()
        v[100:190] = float("nan") if k != "b" else float("inf")
        d[k] = v
    y, s = _fwd(d, cu)
    assert torch.equal(y[:100], y0[:100]) and torch.equal(y[190:], y0[190:])
    assert torch.equal(s[[0, 2]], s0[[0, 2]])


def test_c_entry_leaves_rows_in_no_sequence():
    lib = kda.library()
    d, _ = _make([90], 2, 1, 64, 64, torch.bfloat16, seed=5, init=False, strides=False)
    cu = torch.tensor([7, 7, 60, 81], dtype=torch.int32, device="cuda")
    mark = 2.0 ** 40
    for flags in (0, kda.KDA_ZERO_REST):
        y = torch.full((90, 2, 64), mark, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        rc = lib.kda_ssm_chunk_fwd(d["x"].data_ptr(), 128, d["dt"].data_ptr(), 2, d["A_log"].data_ptr(), d["b"].data_ptr(),
                                   64, d["c"].data_ptr(), 64, None, None, None, cu.data_ptr(), 3, None, y.data_ptr(), 90, 1,
                                   2, 64, 64, flags, 1, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
        assert rc == kda.KDA_OK
        torch.cuda.synchronize()
        rest = torch.cat([y[:7], y[81:]])
        assert bool((rest == (0 if flags else mark)).all()) and not bool((y[7:81] == mark).any())


@pytest.mark.parametrize("cu", [[0, 500, 200, 990], [-7, 5, 5, 10000], [9, 2, -3, 400], [600, 700, 800, 900]])
def test_malformed_offsets_stay_in_bounds(cu):
    d, _ = _make([300, 350, 350], 2, 1, 64, 64, torch.bfloat16, seed=6)
    y, f = _fwd(d, torch.tensor(cu, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert y.shape == d["x"].shape and f.shape == d["state"].shape


def test_no_tokens():
    d, cu = _make([0, 0], 2, 1, 64, 64, torch.bfloat16, seed=7)
    y, f = _fwd(d, cu)
    assert y.shape == (0, 2, 64) and torch.equal(f, d["state"])
    f = _fwd(dict({k: (v.unflatten(0, (2, 0)) if k in TOKEN else v) for k, v in d.items()}), None)[1]
    assert torch.equal(f, d["state"])


def test_wide_token_strides():
    """Token strides at the limit of 2^24 elements: element offsets pass 32 bits."""
    T, ld = 200, 1 << 24
    d, cu = _make([T], 1, 1, 32, 32, torch.bfloat16, seed=8, strides=False)
    buf = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda")
    wide = dict(d)
    at = 0
    for k in ("x", "b", "c"):
        v = buf[at:].as_strided((T, 1, 32), (ld, 32, 1))
        v.copy_(d[k])
        wide[k] = v
        at += 64
    a, b = _fwd(d, cu), _fwd(wide, cu)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_repeats_bit_for_bit_on_a_side_stream_and_in_a_graph():
    d, cu = _make([1500, 3, 700], 2, 1, 128, 64, torch.bfloat16, seed=10)
    pool = torch.zeros(3, 2, 128, 64, device="cuda")

    def both():
        y, f = _fwd(d, cu)
        pool.copy_(f)
        o = kda.kda_ssm_step(d["x"][:3], d["dt"][:3], d["A_log"], d["b"][:3], d["c"][:3], pool, d["D"], d["dt_bias"])
        return y, f, o, pool

    ref = [t.clone() for t in both()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [t.clone() for t in both()]
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
        assert all(torch.equal(a, b) for a, b in zip([t.clone() for t in both()], ref))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rate_past_floats(dtype):
    """exp(A_log) above every float, D_t below: their product is 0 (float64: e^90 e^-200), the decay
    1, and the tokens add nothing: the states come back and y = S^T c + D x."""
    HV, H, K, V, L = 2, 1, 32, 32, 70
    d, cu = _make([L], HV, H, K, V, DT[dtype], seed=11, bias=False)
    d["A_log"] = torch.full_like(d["A_log"], 90.0)
    d["dt"] = torch.full_like(d["dt"], -200.0)
    y, final = _fwd(d, cu)
    _check(d, cu, [L], y, final, dtype)
    assert torch.equal(final, d["state"])
    pool = d["state"].clone()
    out = kda.kda_ssm_step(d["x"][:1].contiguous(), d["dt"][:1], d["A_log"], d["b"][:1].contiguous(),
                           d["c"][:1].contiguous(), pool, d["D"], None)
    assert torch.equal(pool, d["state"]) and bool(torch.isfinite(out).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_tokens(dtype):
    """dt = -inf masks a token: its decay is 1 and it adds nothing, so the states and the other rows
    are those of the sequence with D_t = 0 there, over tiles and segments that are masked whole."""
    HV, H, K, V, L = 2, 1, 64, 64, 700
    d, cu = _make([L], HV, H, K, V, DT[dtype], seed=12)
    mask = torch.rand(L, generator=torch.Generator().manual_seed(13)) < 0.3
    mask[100:420] = True
    d["dt"][mask.cuda()] = float("-inf")
    _check(d, cu, [L], *_fwd(d, cu), dtype)
    d["dt"][:] = float("-inf")
    y, final = _fwd(d, cu)
    _check(d, cu, [L], y, final, dtype)
    assert torch.equal(final, d["state"])


def test_nan_rate_is_not_hidden():
    d, cu = _make([70], 2, 1, 32, 32, torch.bfloat16, seed=14)
    d["A_log"][1] = float("nan")
    y, final = _fwd(d, cu)
    assert bool(torch.isnan(final[0, 1]).all()) and bool(torch.isfinite(final[0, 0]).all())
    assert bool(torch.isfinite(y[:, 0]).all())
    pool = d["state"].clone()
    kda.kda_ssm_step(d["x"][:1].contiguous(), d["dt"][:1], d["A_log"], d["b"][:1].contiguous(),
                     d["c"][:1].contiguous(), pool, d["D"], d["dt_bias"])
    assert bool(torch.isnan(pool[0, 1]).all()) and bool(torch.isfinite(pool[0, 0]).all())
