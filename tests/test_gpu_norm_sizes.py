"""Norms and packing at sizes that read past the caches (a call that moves more than 256 MiB).

A row's outputs do not depend on the other rows, and both forms compute them in the same order, so
they equal those of the same rows in calls that move less, bit for bit (those are compared with the
oracle elsewhere). A sum over rows is compared with the float64 sum of the smaller calls' sums. A term
carries 200 + 4 max|gate| units of 2^-24 (test_gpu_norm's bound; for dscale 130 more, the error of
dresidual) and is added at most rows / 768 + 1 times in a thread, 48 in a slice of the 768 workgroups and 16
over the slices, so each side is within the sum of these units of the sum of absolute terms, taken here
in float64."""

import pytest
import torch

import gated_delta_rule_67_amd as kda
from tests.helpers import log

pytestmark = pytest.mark.gpu

MIB256 = 1 << 28
U = 2.0 ** -24
EPS = 1e-6
TYPES = [(torch.bfloat16, 40001), (torch.float32, 20001)]  # rows of 1024: 82 MB a tensor
D, CHUNK = 1024, 3001  # rows of the smaller calls (24.6 MB a tensor at most)


def _rows(n, dtype, pad=0):
    t = torch.randn(n, D + pad, device="cuda").to(dtype)
    return t[:, pad:]


def _units(n):
    return n / 768 + 1 + 48 + 16 + 200


def _part(v, rows):
    return tuple(t[rows] for t in v) if isinstance(v, tuple) else None if v is None else v[rows]


def _value(v):
    return kda.kda_checkpoint_unpack(*v, torch.float32).double() if isinstance(v, tuple) else v.double()


def _same(n, call, tensors, sums=()):
    """call(*tensors) against calls on CHUNK rows at a time; `sums`: (output index, sum of absolute terms)."""
    whole = call(*tensors)
    index = {i for i, _ in sums}
    total = {i: 0.0 for i in index}
    for first in range(0, n, CHUNK):
        rows = slice(first, min(first + CHUNK, n))
        for i, v in enumerate(call(*(_part(t, rows) for t in tensors))):
            if i in index:
                total[i] = total[i] + v.double()
            else:
                assert torch.equal(whole[i][rows].view(torch.uint8), v.view(torch.uint8)), f"output {i}, rows from {first}"
    for i, terms in sums:
        ratio = float(((whole[i].double() - total[i]).abs() / (2 * terms)).max())
        log(f"    sum {i}: worst |err| / tolerance {ratio:.3f}")
        assert ratio <= 1.0


@pytest.mark.parametrize("dtype,n", TYPES)
@pytest.mark.parametrize("pad", [0, 8])
def test_forward(dtype, n, pad):
    torch.manual_seed(n + pad)
    w, s = torch.randn(D, device="cuda"), torch.randn(D, device="cuda")
    x, r, z = _rows(n, dtype, pad), _rows(n, dtype), _rows(n, dtype, pad)
    assert 4 * n * D * x.element_size() > MIB256
    _same(n, lambda x, r: kda.kda_prenorm_fwd(x, w, r, s, eps=EPS), (x, r))
    _same(n, lambda x, z, r: (kda.kda_postnorm_fwd(x, w, z, r, s, eps=EPS),), (x, z, r))
    _same(n, lambda x, z, r: (kda.kda_postnorm_fwd(x, w, z, r, s, activation="silu", eps=EPS),), (x, z, r))


def test_forward_per_head():
    """Rows of 128, 16 side by side of a token, as slices of the rows of a token."""
    n, G = 33001, 16
    torch.manual_seed(n)
    w = torch.randn(128, device="cuda")
    x, z = (torch.randn(n, G * 128 + 8, device="cuda").to(torch.bfloat16)[:, 8:].unflatten(1, (G, 128)) for _ in range(2))
    assert 3 * x.numel() * 2 > MIB256
    _same(n, lambda x, z: (kda.kda_postnorm_fwd(x, w, z, eps=EPS),), (x, z))


@pytest.mark.parametrize("dtype,n", TYPES)
@pytest.mark.parametrize("packed", [False, True])
def test_in_front_backward(dtype, n, packed):
    torch.manual_seed(n + 1)
    w, s = torch.randn(D, device="cuda"), torch.randn(D, device="cuda")
    h, dy, dh, x = _rows(n, dtype), _rows(n, dtype, 8), _rows(n, dtype), _rows(n, dtype)
    if packed:
        h, x = kda.kda_checkpoint_pack(h), kda.kda_checkpoint_pack(x)
    # dy, dh, dresidual, dx; h and x at 33 bytes for 32 elements, or as they are
    assert n * D * (4 * dy.element_size() + 2 * (33 / 32 if packed else dy.element_size())) > MIB256
    v, e = _value(h), _units(n) * U
    inv = (v.pow(2).mean(-1, keepdim=True) + EPS).rsqrt()
    nv, inner = (v * inv).abs(), (w.double() * dy.double()).abs()
    dweight = e * (dy.double().abs() * nv).sum(0)
    T = inv * (inner + nv * (inner * nv).mean(-1, keepdim=True)) + dh.double().abs()
    dscale = (e + 130 * U) * (_value(x).abs() * T).sum(0)
    del v, inv, nv, inner, T
    _same(n, lambda h, dy, dh, x: kda.kda_prenorm_bwd(h, w, dy, dh, x, s, eps=EPS), (h, dy, dh, x), ((2, dweight), (3, dscale)))


@pytest.mark.parametrize("dtype,n", TYPES)
@pytest.mark.parametrize("packed", [False, True])
def test_behind_backward(dtype, n, packed):
    torch.manual_seed(n + 2)
    w, s = torch.randn(D, device="cuda"), torch.randn(D, device="cuda")
    x, dy, z = _rows(n, dtype), _rows(n, dtype, 8), _rows(n, dtype)
    if packed:
        x, z = kda.kda_checkpoint_pack(x), kda.kda_checkpoint_pack(z)
    assert n * D * (3 * dy.element_size() + 2 * (33 / 32 if packed else dy.element_size())) > MIB256
    v, gate = _value(x), _value(z)
    e = (_units(n) + 4 * float(gate.abs().max())) * U
    terms = (v * (v.pow(2).mean(-1, keepdim=True) + EPS).rsqrt()).abs() * dy.double().abs() * torch.sigmoid(gate)
    dweight, dscale = e * (terms * s.double().abs()).sum(0), e * (terms * w.double().abs()).sum(0)
    del v, gate, terms
    _same(n, lambda x, dy, z: kda.kda_postnorm_bwd(x, w, dy, z, s, eps=EPS), (x, dy, z), ((2, dweight), (3, dscale)))


@pytest.mark.parametrize("dtype,n", [(torch.bfloat16, 90001), (torch.float32, 53001)])
@pytest.mark.parametrize("pad", [0, 8])
def test_packing(dtype, n, pad):
    torch.manual_seed(n)
    x = _rows(n, dtype, pad)
    assert n * D * (x.element_size() + 33 / 32) > MIB256
    _same(n, kda.kda_checkpoint_pack, (x,))
    codes, scales = kda.kda_checkpoint_pack(x)
    _same(n, lambda c, s: (kda.kda_checkpoint_unpack(c, s, dtype),), (codes, scales))
