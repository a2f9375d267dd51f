"""Refusals of the norms, the gated linear recurrence and the checkpoints, without a GPU: validation
returns before any HIP call, and the binding refuses what it can see."""

import ctypes
import os

import pytest
import torch

import gated_delta_rule_67_amd as kda

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails validation
INV, UNS = kda.KDA_ERR_INVALID, kda.KDA_ERR_UNSUPPORTED
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.library_path):
        pytest.skip("libkda.so not built")
    return kda.library()


NORM_BAD = [
    (dict(x=None), INV), (dict(w=None), INV), (dict(y=None), INV), (dict(T=-1), INV), (dict(G=0), INV), (dict(D=0), INV),
    (dict(sx=63), INV), (dict(eps=0.0), INV), (dict(eps=-1.0), INV), (dict(eps=NAN), INV), (dict(eps=INF), INV),
    (dict(dtype=2), INV), (dict(D=8193, sx=8193, sr=8193, sg=8193), UNS), (dict(T=(1 << 30) + 1), UNS),
    (dict(T=1 << 30, G=2, sx=128, sr=128, sg=128), UNS),
]


@pytest.mark.parametrize("bad,rc", NORM_BAD + [(dict(r=FAKE, sr=3), INV)])
def test_prenorm_fwd_refuses(lib, bad, rc):
    a = dict(x=FAKE, sx=64, r=None, sr=64, w=FAKE, y=FAKE, T=4, G=1, D=64, eps=1e-6, dtype=1)
    a.update(bad)
    assert lib.kda_prenorm_fwd(a["x"], a["sx"], a["r"], a["sr"], a["w"], None, a["y"], None, a["T"], a["G"], a["D"], a["eps"],
                               a["dtype"], None) == rc


@pytest.mark.parametrize("bad,rc", NORM_BAD + [(dict(g=FAKE, sg=3), INV), (dict(r=FAKE, sr=3), INV), (dict(flags=2), INV)])
def test_postnorm_fwd_refuses(lib, bad, rc):
    a = dict(x=FAKE, sx=64, g=None, sg=64, r=None, sr=64, w=FAKE, y=FAKE, T=4, G=1, D=64, eps=1e-6, flags=0, dtype=1)
    a.update(bad)
    assert lib.kda_postnorm_fwd(a["x"], a["sx"], a["w"], a["g"], a["sg"], a["r"], a["sr"], None, a["y"], a["T"], a["G"],
                                a["D"], a["eps"], a["flags"], a["dtype"], None) == rc


BWD_BAD = [
    (dict(v=None), INV), (dict(w=None), INV), (dict(dy=None), INV), (dict(out=None), INV), (dict(sv=3), INV), (dict(sdy=3), INV),
    (dict(k=FAKE, more=None), INV), (dict(k=FAKE, sk=3), INV), (dict(vs=FAKE, k=FAKE), INV), (dict(ks=FAKE, k=FAKE), INV),
    (dict(vs=FAKE, D=48, sdy=48), UNS), (dict(eps=0.0), INV), (dict(dtype=7), INV), (dict(ws=None), INV), (dict(ws_bytes=8), INV),
    (dict(ws=ctypes.c_void_p(0x1010)), INV), (dict(D=9000, sv=9000, sdy=9000), UNS),
]


@pytest.mark.parametrize("bad,rc", BWD_BAD)
def test_prenorm_bwd_refuses(lib, bad, rc):
    a = dict(v=FAKE, vs=None, sv=64, w=FAKE, dy=FAKE, sdy=64, k=None, ks=None, sk=64, out=FAKE, more=FAKE, T=4, D=64, eps=1e-6,
             dtype=1, ws=FAKE, ws_bytes=1 << 30)
    a.update(bad)
    scale = FAKE if a["k"] else None
    assert lib.kda_prenorm_bwd(a["v"], a["vs"], a["sv"], a["w"], a["dy"], a["sdy"], None, 0, a["k"], a["ks"], a["sk"], scale,
                               a["out"], a["more"], FAKE, None, a["T"], 1, a["D"], a["eps"], a["dtype"], a["ws"], a["ws_bytes"],
                               None) == rc
    if a["k"] is None and rc == INV and not bad.keys() & {"v"}:
        assert lib.kda_prenorm_bwd(FAKE, None, 64, FAKE, FAKE, 64, None, 0, None, None, 64, FAKE, FAKE, FAKE, FAKE, None, 4, 1, 64,
                                   1e-6, 1, FAKE, 1 << 30, None) == INV  # a scale without x


@pytest.mark.parametrize("bad,rc", BWD_BAD + [(dict(flags=4), INV)])
def test_postnorm_bwd_refuses(lib, bad, rc):
    a = dict(v=FAKE, vs=None, sv=64, w=FAKE, dy=FAKE, sdy=64, k=None, ks=None, sk=64, out=FAKE, more=FAKE, T=4, D=64, eps=1e-6,
             flags=0, dtype=1, ws=FAKE, ws_bytes=1 << 30)
    a.update(bad)
    assert lib.kda_postnorm_bwd(a["v"], a["vs"], a["sv"], a["w"], a["k"], a["ks"], a["sk"], a["dy"], a["sdy"], None, a["out"],
                                a["more"], FAKE, None, a["T"], 1, a["D"], a["eps"], a["flags"], a["dtype"], a["ws"],
                                a["ws_bytes"], None) == rc


@pytest.mark.parametrize("bad,rc", [
    (dict(x=None), INV), (dict(codes=None), INV), (dict(scales=None), INV), (dict(T=-1), INV), (dict(D=0), INV),
    (dict(D=48, sx=48), UNS), (dict(sx=63), INV), (dict(dtype=2), INV), (dict(codes=ctypes.c_void_p(0x1004)), INV),
    (dict(T=1 << 30, D=64), UNS), (dict(T=(1 << 30) + 1, D=32), UNS)])
def test_checkpoint_refuses(lib, bad, rc):
    a = dict(x=FAKE, sx=64, codes=FAKE, scales=FAKE, T=4, D=64, dtype=1)
    a.update(bad)
    assert lib.kda_checkpoint_pack(a["x"], a["sx"], a["codes"], a["scales"], a["T"], a["D"], a["dtype"], None) == rc
    if "sx" not in bad or "D" in bad:
        assert lib.kda_checkpoint_unpack(a["codes"], a["scales"], a["x"], a["T"], a["D"], a["dtype"], None) == rc


GLR_BAD = [
    (dict(x=None), INV), (dict(r=None), INV), (dict(A=None), INV), (dict(N=0), INV), (dict(T=-1), INV), (dict(T=65), INV),
    (dict(D=0), INV), (dict(sx=63), INV), (dict(sr=63), INV), (dict(i=FAKE, si=3), INV), (dict(flags=1), INV), (dict(flags=8), INV),
    (dict(dtype=2), INV), (dict(N=1 << 18, T=1 << 18), UNS), (dict(D=(1 << 20) + 1), UNS), (dict(T=(1 << 30) + 2), UNS),
    (dict(T=1 << 30, D=64), UNS), (dict(N=1 << 17, T=0, D=1 << 14, sx=1 << 14, sr=1 << 14, sdy=1 << 14), UNS),
    (dict(sx=(1 << 24) + 1), UNS), (dict(i=FAKE, si=(1 << 24) + 1), UNS), (dict(T=4096, ws=None), INV), (dict(T=4096, ws_bytes=8), INV),
    (dict(ws=ctypes.c_void_p(0x1010)), INV),
]


@pytest.mark.parametrize("bad,rc", GLR_BAD + [(dict(y=None), INV)])
def test_glr_fwd_refuses(lib, bad, rc):
    a = dict(x=FAKE, sx=64, r=FAKE, sr=64, A=FAKE, i=None, si=64, N=2, y=FAKE, T=64, D=64, flags=4, dtype=1, ws=FAKE, ws_bytes=1 << 40)
    a.update(bad)
    assert lib.kda_glr_fwd(a["x"], a["sx"], a["r"], a["sr"], a["A"], None, a["i"], a["si"], None, None, a["N"], None, a["y"], None,
                           a["T"], a["D"], a["flags"], a["dtype"], a["ws"], a["ws_bytes"], None) == rc


@pytest.mark.parametrize("bad,rc", GLR_BAD + [
    (dict(dy=None), INV), (dict(sdy=3), INV), (dict(sdy=1 << 25), UNS), (dict(dx=None), INV), (dict(dr=None), INV), (dict(i=FAKE, di=None), INV),
    (dict(xs=FAKE), INV), (dict(xs=FAKE, rs=FAKE, i=FAKE), INV), (dict(rs=FAKE), INV),
    (dict(xs=FAKE, rs=FAKE, D=48, sdy=48), UNS)])
def test_glr_bwd_refuses(lib, bad, rc):
    a = dict(x=FAKE, xs=None, sx=64, r=FAKE, rs=None, sr=64, A=FAKE, i=None, si=64, N=2, dy=FAKE, sdy=64, dx=FAKE, dr=FAKE, di=FAKE,
             T=64, D=64, flags=4, dtype=1, ws=FAKE, ws_bytes=1 << 40)
    a.update(bad)
    assert lib.kda_glr_bwd(a["x"], a["xs"], a["sx"], a["r"], a["rs"], a["sr"], a["A"], None, a["i"], None, a["si"], None, None,
                           a["N"], a["dy"], a["sdy"], None, None, a["dx"], a["dr"], a["di"], FAKE, None, None, a["T"], a["D"],
                           a["flags"], a["dtype"], a["ws"], a["ws_bytes"], None) == rc


@pytest.mark.parametrize("bad,rc", [
    (dict(x=None), INV), (dict(r=None), INV), (dict(A=None), INV), (dict(pool=None), INV), (dict(y=None), INV), (dict(B=0), INV),
    (dict(nslots=0), INV), (dict(slots=None, nslots=3), INV), (dict(sx=8), INV), (dict(flags=2), INV), (dict(dtype=3), INV),
    (dict(D=1 << 21, sx=1 << 21, sr=1 << 21), UNS), (dict(B=1 << 22), UNS)])
def test_glr_step_refuses(lib, bad, rc):
    a = dict(x=FAKE, sx=512, r=FAKE, sr=512, A=FAKE, pool=FAKE, slots=FAKE, nslots=8, y=FAKE, B=4, D=512, flags=4, dtype=1)
    a.update(bad)
    assert lib.kda_glr_step(a["x"], a["sx"], a["r"], a["sr"], a["A"], None, None, 0, a["pool"], a["slots"], a["nslots"], a["y"],
                            a["B"], a["D"], a["flags"], a["dtype"], None) == rc


def test_workspaces(lib):
    fwd, bwd, norm = lib.kda_glr_fwd_workspace_size, lib.kda_glr_bwd_workspace_size, lib.kda_norm_bwd_workspace_size
    assert fwd(0, 64) == 0 and fwd(1, 64) == 0 and fwd(1, 0) == 0 and fwd(-1, 64) == 0
    assert fwd(8192, 64) >= 8192 // 128 * 64 * 8 and fwd(8192, 65) % 256 == 0
    assert bwd(32, 64, 1) == 2 * 64 * 4 and bwd(32, 64, 0) == 3 * 64 * 4  # one tile: partial sums (and a state)
    assert bwd(8192, 64, 0) >= bwd(8192, 64, 1) + 8192 // 64 * 64 * 4
    assert norm(0, 1, 64) == 0 and norm(1, 1, 64) == 512 and norm(1 << 20, 16, 128) <= 2048 * 2 * 128 * 4
    assert norm(4, 1, 8193) == 0


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(2, 8, 32), torch.zeros(32)
    for call in (lambda: kda.kda_prenorm_fwd(x, w), lambda: kda.kda_postnorm_fwd(x, w, x), lambda: kda.kda_prenorm_bwd(x, w, x),
                 lambda: kda.kda_postnorm_bwd(x, w, x), lambda: kda.kda_checkpoint_pack(x),
                 lambda: kda.kda_checkpoint_unpack(x.to(torch.float8_e4m3fn), x.to(torch.uint8)),
                 lambda: kda.kda_glr_fwd(x, x, w), lambda: kda.kda_glr_bwd(x, x, w, x), lambda: kda.kda_glr_step(x[0], x[0], w, x[0])):
        with pytest.raises(ValueError):
            call()
