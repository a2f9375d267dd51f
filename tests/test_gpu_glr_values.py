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
