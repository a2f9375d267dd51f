"""Calls at the limits that the recurrence's documentation names."""

import pytest
import torch

import gated_delta_rule_67_amd as kda

FAKE = 0x1000  # never dereferenced


@pytest.mark.gpu
@pytest.mark.parametrize("D,B", [(256, 1 << 22), (512, (1 << 22) - 1)])
def test_step_of_as_many_requests_as_are_allowed(D, B):
    """B ceil(D / 256) < 2^23, at widths of whole pieces of 256 channels. Requests without a slot give zeros, the
    others (the last one among them) what a call of their own gives."""
    x = torch.empty(B, D, dtype=torch.bfloat16, device="cuda")
    some = torch.tensor([0, 1, 77, B // 2, B - 2, B - 1], device="cuda")
    x[some] = torch.randn(6, D, device="cuda").to(x.dtype)
    A, pool = torch.randn(D, device="cuda"), torch.randn(8, D, device="cuda")
    slots = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    at = torch.tensor([3, 0, 7, 1, 5, 2], dtype=torch.int32, device="cuda")
    slots[some] = at
    few = pool.clone()
    ref = kda.kda_glr_step(x[some], x[some], A, few, None, x[some], at)
    y = kda.kda_glr_step(x, x, A, pool, None, x, slots)
    assert torch.equal(y[some], ref) and torch.equal(pool, few)
    y[some] = 0
    assert not y.view(torch.int32).any()


@pytest.mark.parametrize("D,B", [(256, 1 << 23), (257, 1 << 22), (512, 1 << 22)])
def test_step_of_more_requests_is_refused(D, B):
    assert kda.library().kda_glr_step(FAKE, D, FAKE, D, FAKE, None, None, 0, FAKE, FAKE, 8, FAKE, B, D, 0, 1, None) \
        == kda.KDA_ERR_UNSUPPORTED
