"""kda_checkpoint_pack / kda_checkpoint_unpack against the oracle's table of codes: equal, bit for bit
(scales are powers of two, so a code is rounded once and a value not at all)."""

import numpy as np
import pytest
import torch

import gated_delta_rule_67_amd as kda
from oracle import checkpoint_pack, checkpoint_unpack
from tests.helpers import to64

pytestmark = pytest.mark.gpu


def _same(x):
    codes, scales = kda.kda_checkpoint_pack(x)
    assert codes.shape == x.shape and codes.dtype is torch.float8_e4m3fn and scales.dtype is torch.uint8
    ref, byte = checkpoint_pack(to64(x))
    got = codes.view(torch.uint8).cpu().numpy()
    nan = (ref & 127) == 127
    assert np.array_equal(scales.cpu().numpy(), byte)
    assert np.array_equal(got[~nan], ref[~nan]) and np.all((got[nan] & 127) == 127)
    values = checkpoint_unpack(ref, byte)
    assert np.array_equal(to64(kda.kda_checkpoint_unpack(codes, scales, torch.float32)), values.astype(np.float32), equal_nan=True)
    bf = torch.from_numpy(values).to(torch.float32).to(torch.bfloat16)  # rounds what is below bf16's range
    assert torch.equal(torch.nan_to_num(kda.kda_checkpoint_unpack(codes, scales).cpu()), torch.nan_to_num(bf))


@pytest.mark.parametrize("shape", [(1, 32), (3, 64), (2, 5, 96), (7, 1056), (129, 2048), (4, 2, 3, 32), (32,)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_values(shape, dtype):
    torch.manual_seed(shape[0])
    x = torch.randn(shape) * 10.0 ** (6 * torch.rand(shape[:-1] + (1,)) - 3)
    _same(x.to(dtype).cuda())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_magnitude(dtype):
    """Blocks whose largest element is at, just under and just over every border, over the whole range."""
    e = torch.arange(-148, 128, dtype=torch.float64)
    top = torch.cat([2.0 ** e * m for m in (1.0, 1.5, 1.75, 1.7578125, 1.9921875)]).clamp(max=3.38e38)
    x = top[:, None] * torch.linspace(-1, 1, 32, dtype=torch.float64)
    x[:, 5], x[:, 6] = top, 2.0 ** -12 * top
    _same(x.float().to(dtype).cuda())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ties_and_values_that_are_not_finite(dtype):
    codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mid = torch.cat([(codes[1:] + codes[:-1]) / 2, codes[:2]])  # 128 values, exact in bf16
    x = mid.reshape(4, 32).repeat(1, 2)
    x[:, 32:] = -x[:, 32:]
    x[:, 0], x[:, 33] = 448.0, -448.0  # the scale is 1 in every block
    x[1, 3], x[1, 40], x[2, 9] = float("inf"), float("nan"), float("-inf")
    x[3, 32:] = float("nan")
    _same(x.to(dtype).cuda())


def test_no_tokens_and_slices():
    codes, scales = kda.kda_checkpoint_pack(torch.empty((0, 64), device="cuda"))
    assert codes.shape == (0, 64) and scales.shape == (0, 2)
    assert kda.kda_checkpoint_unpack(codes, scales).shape == (0, 64)
    wide = torch.randn(50, 3 * 64 + 3, device="cuda").to(torch.bfloat16)
    for x in (wide[:, 3:].unflatten(1, (3, 64)), wide[:, 2:66], wide[::2, :64]):
        for a, b in zip(kda.kda_checkpoint_pack(x), kda.kda_checkpoint_pack(x.contiguous())):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_unaligned_outputs():
    lib = kda.library()
    x = torch.randn(40, 96, device="cuda").to(torch.bfloat16)
    codes, scales = kda.kda_checkpoint_pack(x)
    buf = torch.empty(40 * 96 + 1, dtype=torch.bfloat16, device="cuda")
    assert lib.kda_checkpoint_unpack(codes.data_ptr(), scales.data_ptr(), buf[1:].data_ptr(), 40, 96, 1,
                                     torch.cuda.current_stream().cuda_stream) == kda.KDA_OK
    assert torch.equal(buf[1:].view(40, 96), kda.kda_checkpoint_unpack(codes, scales))


def test_repeats_in_a_graph():
    x = torch.randn(700, 320, device="cuda").to(torch.bfloat16)
    ref = kda.kda_checkpoint_unpack(*kda.kda_checkpoint_pack(x)).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kda.kda_checkpoint_unpack(*kda.kda_checkpoint_pack(x))
    for _ in range(3):
        got.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, ref) and torch.equal(kda.kda_checkpoint_unpack(*kda.kda_checkpoint_pack(x)), ref)
