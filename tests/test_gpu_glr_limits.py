"""Calls at and past the limits that the recurrence's documentation names, and sizes past 32 bits."""

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


BIG = 1 << 32


def test_sizes_past_32_bits_are_refused_by_the_checks():
    """ctypes passes on an int's low 32 bits: such a size must not reach it."""
    huge = torch.empty(BIG + 1, 0, 8, device="meta")
    for call in (lambda: kda._sequences(huge, None, 3, -1), lambda: kda._slots(None, 3, BIG + 5, -1),
                 lambda: kda._sequences(torch.empty(5, 8, device="meta"), torch.empty(BIG + 2, dtype=torch.int32, device="meta"), 3, -1),
                 lambda: kda._glr_params(BIG + 64, None, None, -1)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_sizes_past_32_bits_are_refused():
    flat = torch.empty(BIG + 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        kda.kda_checkpoint_pack(flat)
    with pytest.raises(ValueError):
        kda.kda_checkpoint_unpack(flat[:BIG // 2 + 32].view(torch.float8_e4m3fn), flat[:BIG // 64 + 1].view(torch.uint8))
    del flat
    one, pool = torch.ones(1, 1, device="cuda"), torch.empty(BIG + 5, 1, device="cuda")
    with pytest.raises(ValueError):
        kda.kda_glr_step(one, one, one[0], pool, slots=torch.tensor([7], dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        kda.kda_glr_fwd(torch.empty(BIG + 1, 0, 1, device="cuda"), torch.empty(BIG + 1, 0, 1, device="cuda"), one[0])
