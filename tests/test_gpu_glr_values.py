"""The recurrence's gate where its input and its bias are large.

Tolerance, with u = 2^-24 and z = gate_x + dt_bias: the sum is rounded once (|z| u), log2 e is a float (0.3 u) and
its product with z is rounded once (u), so that the softplus, whose relative error from an error dz of its
input is at most dz, carries 2.3 |z| u beside the 17 u of test_gpu_glr; no term grows with |dt_bias|. For |z| <= 5 that
is within the (24 + |z|) u of test_gpu_glr's bounds, which are used as they are."""

import numpy as np
import pytest
import torch

import gated_delta_rule_67_amd as kda
from oracle import glr_gates
from tests.helpers import to64
from tests.test_gpu_glr import _check, _make
from tests.test_gpu_norm import U, close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,size", [(torch.float32, 20.0), (torch.float32, 60.0), (torch.float32, 100.0),
                                        (torch.float32, 3000.0), (torch.bfloat16, 60.0), (torch.bfloat16, 100.0)])
def test_biases_that_cancel(dtype, size):
    """Forward and backward, with biases of either sign that leave |z| <= 5 (of bf16 inputs, too: half a step is
    0.25 at 110)."""
    d = _make([1] * 40 + [0, 3, 70], 64, dtype, int(size))
    g = torch.Generator().manual_seed(int(size))
    bias = size * (1 + 0.1 * torch.rand(64, generator=g)) * torch.where(torch.arange(64) % 2 == 0, 1.0, -1.0)
    z = torch.randn(d["x"].shape, generator=g).clamp(-4, 4)
    d.update(dt_bias=bias.cuda(), gate_x=(z - bias).to(dtype).cuda(), A_log=0.5 * torch.randn(64, generator=g).cuda())
    assert float((d["gate_x"].double() + d["dt_bias"].double()).abs().max()) <= 5
    _check(d, dtype)


@pytest.mark.parametrize("bias", [0.0, -40.0, 33.3])
def test_far_negative_gates(bias):
    """One token from a state of zero: y = sqrt(1 - a^2), within half the log decay's error and 20 u."""
    z = torch.linspace(-85.0, -1.0, 400)
    r = (z - bias)[:, None].cuda()
    A, b = torch.tensor([0.7], device="cuda"), torch.tensor([bias], device="cuda")
    pool = torch.zeros(400, 1, device="cuda")
    y = kda.kda_glr_step(torch.ones_like(r), r, A, pool, b)
    zz, _, _, w, _ = glr_gates(to64(r), to64(A), to64(b))
    close(y, w, np.abs(w) * ((17 + 2.3 * np.abs(zz)) / 2 + 20) * U, "y")
    assert torch.equal(y, pool)


@pytest.mark.parametrize("lengths,D,dtype,packed", [([65], 64, "bf16", False), ([121, 200], 65, "f32", False),
                                                    ([5000, 3192], 2048, "bf16", False), ([65], 64, "bf16", True),
                                                    ([3000, 1000], 256, "bf16", True)])
def test_no_wait_gives_up(lengths, D, dtype, packed):
    """The second word of a workspace tells of waits that gave up: every call leaves it as it was, whatever the rest
    of the workspace held."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    d, lib, s = _make(lengths, D, dt, D), kda.library(), torch.cuda.current_stream().cuda_stream
    T, N = sum(lengths), len(lengths)
    n, m, k = lib.kda_glr_fwd_workspace_size(T, D), lib.kda_glr_bwd_workspace_size(T, D, 0), lib.kda_glr_bwd_workspace_size(T, D, 1)
    y, dx, dr, di = (torch.empty_like(d["x"]) for _ in range(4))
    states, dA = torch.empty((T + 63) // 64, D, device="cuda"), torch.empty(D, device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    held = [kda.kda_checkpoint_pack(d[v]) if packed else (d[v], None) for v in ("x", "gate_x", "in_gate")]
    kept = [(p(a), None if b is None else p(b), D) for a, b in held]
    for fill in (0, 0xff, 0x5a):
        ws = torch.full((max(n, m, k) // 4,), fill * 0x01010101 - (1 << 32 if fill > 127 else 0), dtype=torch.int32, device="cuda")
        for clear in (0, 7):
            ws[1] = clear
            assert lib.kda_glr_fwd(p(d["x"]), D, p(d["gate_x"]), D, p(d["A_log"]), p(d["dt_bias"]), p(d["in_gate"]), D, p(d["init"]),
                                   p(d["cu"]), N, None, p(y), p(states), T, D, 4, int(dt is torch.bfloat16), p(ws), n, s) == 0
            assert int(ws[1]) == clear
            for have, size in ((None, m),) if packed else ((None, m), (p(states), k)):
                assert lib.kda_glr_bwd(*kept[0], *kept[1], p(d["A_log"]), p(d["dt_bias"]), *kept[2], p(d["init"]), p(d["cu"]), N,
                                       p(d["dy"]), D, None, have, p(dx), p(dr), p(di), p(dA), None, None, T, D, 4,
                                       int(dt is torch.bfloat16), p(ws), size, s) == 0
                assert int(ws[1]) == clear
    assert bool(torch.isfinite(dA).all())


def test_states_beside_checkpoints():
    """Block states of a forward pass over the values that checkpoints stand for give the gradients of a call that
    computes them again, up to their rounding on the way (the same values in float32)."""
    d = _make([300, 70], 96, torch.float32, 9, rate=-4.0)
    kept = [kda.kda_checkpoint_pack(d[k]) for k in ("x", "gate_x", "in_gate")]
    x, r, i = (kda.kda_checkpoint_unpack(*t, torch.float32) for t in kept)
    states = kda.kda_glr_fwd(x, r, d["A_log"], d["dt_bias"], i, d["init"], d["cu"], output_block_states=True)[2]
    args = (d["A_log"], d["dy"], d["dt_bias"])
    rest = (d["init"], d["dfinal"], d["cu"])
    given = kda.kda_glr_bwd(kept[0], kept[1], *args, kept[2], *rest, block_states=states)
    again = kda.kda_glr_bwd(kept[0], kept[1], *args, kept[2], *rest)
    plain = kda.kda_glr_bwd(x, r, *args, i, *rest, block_states=states)
    for a, b, c in zip(given, again, plain):
        assert torch.equal(a, c)
        assert float((a - b).abs().max()) <= 400 * 60 * U * float(c.abs().max())


@pytest.mark.parametrize("gate", [-200.0, -87.0, -60.0, -3.0])
def test_large_inputs_under_small_weights(gate):
    """|x| up to 2^63.9: finite gradients, 0 from a weight of 0; the gate's is that of the oracle."""
    x = torch.tensor([[2.0 ** 63.9, -2.0 ** 63.9, 1.0, 0.0]], device="cuda")
    r, A = torch.full_like(x, gate), torch.tensor([0.3] * 4, device="cuda")
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    dx, dr = kda.kda_glr_bwd(x, r, A, torch.ones_like(x), cu_seqlens=cu)[:2]
    assert bool(torch.isfinite(dx).all() and torch.isfinite(dr).all())
    if gate == -200.0:
        assert not dr.any() and not dx.any()
    elif gate >= -60.0:
        z, _, a, w, _ = glr_gates(to64(r), to64(A))
        ref = np.exp(0.3) * to64(x) * a * a / w / (1 + np.exp(-z))
        # weight, decay and slope within (17 + 2.3 |z|) u each, twice over, and 40 u
        close(dr, ref, np.abs(ref) * (3 * (17 + 2.3 * abs(gate)) + 40) * U, "dgate_x")
