"""Refusals of the convolution, selective scan and slot entry points, without a GPU: validation
returns before any HIP call, and the binding refuses tensors that are not on a GPU."""

import ctypes
import os

import pytest
import torch

import gated_delta_rule_67_amd as kda

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails validation


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.library_path):
        pytest.skip("libkda.so not built")
    return kda.library()


INV, UNS = kda.KDA_ERR_INVALID, kda.KDA_ERR_UNSUPPORTED
CONV_BAD = [
    (dict(x=None), INV), (dict(weight=None), INV), (dict(N=0), INV), (dict(T=-1), INV), (dict(D=0), INV),
    (dict(T=65), INV),                       # T % N without offsets
    (dict(x_stride=63), INV),                # rows overlap
    (dict(dtype=2), INV), (dict(flags=8), INV),
    (dict(W=1), UNS), (dict(W=5), UNS), (dict(D=1 << 21, x_stride=1 << 21), UNS),
    (dict(N=1 << 18, T=1 << 18), UNS),
]


@pytest.mark.parametrize("bad,rc", CONV_BAD + [(dict(y=None), INV)])
def test_conv_fwd_refuses(lib, bad, rc):
    a = dict(x=FAKE, x_stride=64, weight=FAKE, N=2, y=FAKE, T=64, D=64, W=4, flags=1, dtype=1)
    a.update(bad)
    assert lib.kda_conv_fwd(a["x"], a["x_stride"], a["weight"], None, None, None, a["N"], None, a["y"], a["T"],
                            a["D"], a["W"], a["flags"], a["dtype"], None) == rc


@pytest.mark.parametrize("bad,rc", CONV_BAD + [
    (dict(dy=None), INV), (dict(dx=None), INV), (dict(dy_stride=3), INV), (dict(ws=None), INV),
    (dict(ws_bytes=4), INV), (dict(ws=ctypes.c_void_p(0x1010)), INV)])
def test_conv_bwd_refuses(lib, bad, rc):
    a = dict(x=FAKE, x_stride=64, weight=FAKE, N=2, dy=FAKE, dy_stride=64, dx=FAKE, T=64, D=64, W=4, flags=1,
             dtype=1, ws=FAKE, ws_bytes=1 << 30)
    a.update(bad)
    assert lib.kda_conv_bwd(a["x"], a["x_stride"], a["weight"], None, None, None, a["N"], a["dy"], a["dy_stride"],
                            None, a["dx"], None, None, None, a["T"], a["D"], a["W"], a["flags"], a["dtype"],
                            a["ws"], a["ws_bytes"], None) == rc


@pytest.mark.parametrize("bad,rc", [
    (dict(x=None), INV), (dict(pool=None), INV), (dict(y=None), INV), (dict(B=0), INV), (dict(nslots=0), INV),
    (dict(slots=None, nslots=3), INV), (dict(x_stride=8), INV), (dict(W=5), UNS), (dict(B=70000), UNS),
    (dict(dtype=3), INV)])
def test_conv_step_refuses(lib, bad, rc):
    a = dict(x=FAKE, x_stride=64, weight=FAKE, pool=FAKE, slots=FAKE, nslots=8, y=FAKE, B=4, D=64, W=4, dtype=1)
    a.update(bad)
    assert lib.kda_conv_step(a["x"], a["x_stride"], a["weight"], None, a["pool"], a["slots"], a["nslots"], a["y"],
                             a["B"], a["D"], a["W"], 1, a["dtype"], None) == rc


def test_conv_workspace(lib):
    ws = lib.kda_conv_bwd_workspace_size
    assert ws(0, 64, 4, 1) == 0 and ws(64, 64, 9, 1) == 0
    assert ws(4, 64, 4, 1) == 5 * 64 * 4  # one row block: (W + 1) D floats
    assert ws(32768, 6144, 4, 1) <= 128 * 5 * 6144 * 4


SSM_BAD = [
    (dict(x=None), INV), (dict(dt=None), INV), (dict(A_log=None), INV), (dict(b=None), INV), (dict(c=None), INV),
    (dict(y=None), INV), (dict(HV=3), INV), (dict(H=0), INV), (dict(K=0), INV), (dict(V=0), INV), (dict(dtype=2), INV),
    (dict(K=129, sb=258, sc=258), UNS), (dict(V=136, sx=4 * 136), UNS), (dict(sx=255), INV), (dict(sdt=3), INV),
    (dict(sb=100), INV), (dict(sc=-5), INV),
]


@pytest.mark.parametrize("bad,rc", SSM_BAD + [
    (dict(N=0), INV), (dict(T=-1), INV), (dict(T=65), INV), (dict(flags=1), INV), (dict(sx=(1 << 24) + 1), UNS),
    (dict(T=8192, N=1, ws=None), INV), (dict(T=8192, N=1, ws_bytes=8), INV), (dict(ws=ctypes.c_void_p(0x1010)), INV),
    (dict(N=1 << 21, T=1 << 21), UNS)])
def test_ssm_chunk_fwd_refuses(lib, bad, rc):
    a = dict(x=FAKE, sx=256, dt=FAKE, sdt=4, A_log=FAKE, b=FAKE, sb=128, c=FAKE, sc=128, N=2, y=FAKE, T=64, H=2, HV=4,
             K=64, V=64, flags=0, dtype=1, ws=FAKE, ws_bytes=1 << 40)
    a.update(bad)
    assert lib.kda_ssm_chunk_fwd(a["x"], a["sx"], a["dt"], a["sdt"], a["A_log"], a["b"], a["sb"], a["c"], a["sc"], None,
                                 None, None, None, a["N"], None, a["y"], a["T"], a["H"], a["HV"], a["K"], a["V"],
                                 a["flags"], a["dtype"], a["ws"], a["ws_bytes"], None) == rc


@pytest.mark.parametrize("bad,rc", SSM_BAD + [
    (dict(pool=None), INV), (dict(B=0), INV), (dict(nslots=0), INV), (dict(slots=None, nslots=3), INV),
    (dict(B=1 << 28), UNS)])
def test_ssm_step_refuses(lib, bad, rc):
    a = dict(x=FAKE, sx=256, dt=FAKE, sdt=4, A_log=FAKE, b=FAKE, sb=128, c=FAKE, sc=128, pool=FAKE, slots=FAKE, nslots=8,
             y=FAKE, B=4, H=2, HV=4, K=64, V=64, dtype=1)
    a.update(bad)
    assert lib.kda_ssm_step(a["x"], a["sx"], a["dt"], a["sdt"], a["A_log"], a["b"], a["sb"], a["c"], a["sc"], None, None,
                            a["pool"], a["slots"], a["nslots"], a["y"], a["B"], a["H"], a["HV"], a["K"], a["V"],
                            a["dtype"], None) == rc


def test_ssm_workspace(lib):
    ws = lib.kda_ssm_chunk_fwd_workspace_size
    assert ws(1, 256, 0, 1, 1, 64, 64, 1) == 0           # one segment
    assert ws(4, 4 * 8192, 0, 64, 512, 64, 64, 1) == 0   # whole sequences fill the GPU
    one = 16 * (128 * 128 + 1) * 4                       # a boundary's states and decays
    n = ws(1, 8192, 0, 1, 16, 128, 128, 1)
    assert n > 0 and n % 256 == 0 and n // one == 31     # 32 segments of 256 tokens
    assert ws(1, 0, 1, 1, 16, 128, 128, 1) == 0 and ws(3, 8192, 0, 1, 16, 128, 128, 1) == 0
    assert ws(1, 8192, 0, 1, 16, 200, 128, 1) == 0


def _arrays(ptrs, sizes):
    return (ctypes.c_void_p * len(ptrs))(*ptrs), (ctypes.c_size_t * len(sizes))(*sizes)


@pytest.mark.parametrize("bad,rc", [
    (dict(ptrs=[0x1000, None]), INV), (dict(sizes=[16, 0]), INV), (dict(nslots=0), INV), (dict(n=-1), INV),
    (dict(src=None), INV), (dict(dst=None), INV), (dict(npools=-1), INV), (dict(nslots=1 << 19), UNS),
    (dict(sizes=[16, (1 << 40) + 1]), UNS)])
def test_slots_copy_refuses(lib, bad, rc):
    a = dict(ptrs=[0x1000, 0x2000], sizes=[16, 16], npools=2, nslots=4, src=FAKE, dst=FAKE, n=2)
    a.update(bad)
    base, size = _arrays(a["ptrs"], a["sizes"])
    assert lib.kda_slots_copy(base, size, a["npools"], a["nslots"], a["src"], a["dst"], a["n"], None) == rc


@pytest.mark.parametrize("bad,rc", [
    (dict(live=None), INV), (dict(new=None), INV), (dict(count=None), INV), (dict(ws=None), INV),
    (dict(ws_bytes=8), INV), (dict(ws=ctypes.c_void_p(0x1010)), INV), (dict(nslots=1 << 19), UNS)])
def test_slots_compact_refuses(lib, bad, rc):
    a = dict(live=FAKE, new=FAKE, count=FAKE, ws=FAKE, ws_bytes=1 << 20, nslots=4)
    a.update(bad)
    base, size = _arrays([0x1000], [16])
    assert lib.kda_slots_compact(base, size, 1, a["nslots"], a["live"], a["new"], a["count"], a["ws"],
                                 a["ws_bytes"], None) == rc


def test_nothing_to_do_returns_ok(lib):
    base, size = _arrays([0x1000], [16])
    assert lib.kda_slots_copy(base, size, 1, 4, None, None, 0, None) == kda.KDA_OK
    assert lib.kda_slots_copy(None, None, 0, 4, FAKE, FAKE, 3, None) == kda.KDA_OK


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(2, 8, 16), torch.zeros(16, 4)
    for call in (lambda: kda.kda_conv_fwd(x, w), lambda: kda.kda_conv_bwd(x, w, x),
                 lambda: kda.kda_ssm_chunk_fwd(x[..., None], x, w[0], x[..., None], x[..., None]),
                 lambda: kda.kda_ssm_step(x, x[..., 0], w[0], x, x, x[None]),
                 lambda: kda.kda_conv_step(x[:, 0], w, torch.zeros(2, 3, 16)),
                 lambda: kda.kda_slots_copy(x, torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)),
                 lambda: kda.kda_slots_compact([x], torch.ones(2, dtype=torch.bool)),
                 lambda: kda.kda_slots_copy([], torch.zeros(1), torch.zeros(1))):
        with pytest.raises(ValueError):
            call()


def test_token_limit(lib):
    """Sums of a token's index and a tile's or a segment's length stay in 32 bits: T <= 2^30."""
    T = (1 << 30) + 1
    assert lib.kda_conv_fwd(FAKE, 1, FAKE, None, None, None, 1, None, FAKE, T, 1, 4, 1, 1, None) == UNS
    assert lib.kda_conv_bwd(FAKE, 1, FAKE, None, None, None, 1, FAKE, 1, None, FAKE, None, None, None, T, 1, 4, 1, 1,
                            FAKE, 1 << 40, None) == UNS
    assert lib.kda_ssm_chunk_fwd(FAKE, 1, FAKE, 1, FAKE, FAKE, 1, FAKE, 1, None, None, None, None, 1, None, FAKE, T,
                                 1, 1, 1, 1, 0, 1, FAKE, 1 << 40, None) == UNS
    assert lib.kda_conv_bwd_workspace_size(T, 1, 4, 1) == 0
    assert lib.kda_ssm_chunk_fwd_workspace_size(1, T, 0, 1, 1, 1, 1, 1) == 0


def test_launch_limit(lib):
    """A launch holds fewer than 2^32 threads: what needs more is refused before it."""
    def step(B, HV):
        return lib.kda_ssm_step(FAKE, HV, FAKE, HV, FAKE, FAKE, 1, FAKE, 1, None, None, FAKE, FAKE, 1, FAKE, B, 1, HV,
                                1, 1, 1, None)
    assert step(1 << 17, 1 << 6) == UNS      # 2^23 heads of 512 threads
    assert step(1 << 30, 1 << 3) == UNS
    N, HV = 1 << 19, 64                      # one token each, 32 workgroups of 256 threads a sequence
    assert lib.kda_ssm_chunk_fwd_workspace_size(N, N, 0, 1, HV, 1, 64, 1) == 0
    assert lib.kda_ssm_chunk_fwd(FAKE, HV * 64, FAKE, HV, FAKE, FAKE, 1, FAKE, 1, None, None, None, None, N, None, FAKE,
                                 N, 1, HV, 1, 64, 0, 1, None, 0, None) == UNS
