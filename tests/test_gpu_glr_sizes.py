"""kda_glr_fwd / kda_glr_bwd with several tiles for every workgroup, and over dense batches whose
sequences are whole tiles, which take their tiles side by side.

At the large sizes a few columns are compared with the float64 oracle, within the bounds that
test_gpu_glr derives, and every element with the same call on 64 columns at a time: a column's tiles along the
tokens and their order do not depend on how many columns there are, so the results are equal bit for
bit. Those calls have fewer tiles than there are workgroups."""

import numpy as np
import pytest
import torch

import gated_delta_rule_67_amd as kda
from oracle import glr, glr_bwd
from tests.helpers import log, to64
from tests.test_gpu_glr import _bounds, _check, _make
from tests.test_gpu_norm import HALF, U, close

pytestmark = pytest.mark.gpu

TOKENS = ("x", "gate_x", "in_gate", "dy")


def _cut(d, columns):
    """The same inputs on some channels."""
    return {k: v if v is None or k == "cu" else v[..., columns] if k in TOKENS else v[..., columns].contiguous()
            for k, v in d.items()}


def _run(d, dense, packed):
    """{name: output}, token tensors as [tokens, channels]."""
    N = d["cu"].numel() - 1
    shaped = lambda v: v.unflatten(0, (N, -1)) if dense else v  # noqa: E731
    off = None if dense else d["cu"]
    kept = {k: shaped(d[k]) for k in TOKENS}
    if packed:
        kept.update({k: kda.kda_checkpoint_pack(kept[k]) for k in TOKENS[:3]})
        y = f = states = None
    else:
        y, f, states = kda.kda_glr_fwd(kept["x"], kept["gate_x"], d["A_log"], d["dt_bias"], kept["in_gate"], d["init"], off,
                                       output_block_states=True)
    g = kda.kda_glr_bwd(kept["x"], kept["gate_x"], d["A_log"], kept["dy"], d["dt_bias"], kept["in_gate"], d["init"], d["dfinal"],
                        off, block_states=states)
    torch.cuda.synchronize()
    out = dict(zip(("dx", "dr", "di", "dA", "db", "dinit"), g))
    if not packed:
        out.update(y=y, final=f)
    return {k: v.reshape(d["dy"].shape) if k in ("y", "dx", "dr", "di") else v for k, v in out.items()}


def _against_the_oracle(d, got, dtype):
    """All columns of d, whose outputs are got."""
    half, cu = HALF[dtype], d["cu"].cpu().numpy()
    h = {k: None if v is None else to64(v) for k, v in d.items()}
    N, D = len(cu) - 1, h["A_log"].shape[0]
    sums, room = np.zeros((2, D)), np.zeros((2, D))
    for n in range(N):
        t = slice(cu[n], cu[n + 1])
        args = (h["x"][t], h["gate_x"][t], h["A_log"])
        rest = (h["in_gate"][t], h["init"][n])
        b = _bounds(*args, h["dt_bias"], *rest, h["dy"][t], h["dfinal"][n], True)
        r = glr_bwd(*args, h["dy"][t], h["dt_bias"], *rest, h["dfinal"][n])
        for name, ref, tol in (("dx", r[0], b[2]), ("dr", r[1], b[3]), ("di", r[2], b[4])):
            close(got[name][t], ref, half * np.abs(ref) + tol, f"{name} of sequence {n}")
        close(got["dinit"][n], r[5], b[5], "dinitial_state")
        sums += [r[3], r[4]]
        room += [(cu[n + 1] - cu[n]) * U * b[6] + b[7], (cu[n + 1] - cu[n]) * U * b[8] + b[9]]
        if "y" in got:
            y, f = glr(*args, h["dt_bias"], *rest)
            close(got["y"][t], y, half * np.abs(y) + b[0], f"y of sequence {n}")
            close(got["final"][n], f, b[1], "final state")
    close(got["dA"], sums[0], room[0], "dA_log")
    close(got["db"], sums[1], room[1], "ddt_bias")


def _check_wide(d, dtype, dense=False, packed=False):
    D = d["A_log"].numel()
    got = _run(d, dense, packed)
    for c in range(0, D, 64):
        cut = slice(c, min(c + 64, D))
        for name, v in _run(_cut(d, cut), dense, packed).items():
            assert torch.equal(got[name][..., cut], v), f"{name}, columns from {c}"
    if packed:  # the values that the codes stand for
        d = dict(d, **{k: kda.kda_checkpoint_unpack(*kda.kda_checkpoint_pack(d[k]), torch.float32) for k in TOKENS[:3]})
    some = torch.tensor(sorted({0, 1, 63, D // 2, D - 2, D - 1}), device="cuda")
    _against_the_oracle(_cut(d, some), {k: v[..., some] for k, v in got.items()}, dtype)


# tiles forward (120 tokens; 60 from checkpoints) and backward (64), by columns of 128 channels of bf16,
# 64 of float32 or of an odd width, and 256 forward from checkpoints
@pytest.mark.parametrize("lengths,D,dtype,packed", [
    ([5000, 0, 1, 3191], 2048, "bf16", False),    # 69 x 16 forward, 128 x 16 backward
    ([8193], 1030, "f32", False),                 # 69 x 17, 129 x 17
    ([1200, 6000, 999], 1027, "bf16", False),     # 69 x 17, 129 x 17, one channel a lane
    ([3000, 4, 5188], 2048, "bf16", True),        # 137 x 8, 128 x 16
    ([4100, 4092], 1056, "f32", True),            # 137 x 5, 128 x 17
])
def test_several_tiles_a_workgroup(lengths, D, dtype, packed):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    log(f"glr lengths={lengths} D={D} {dtype} packed={packed}")
    _check_wide(_make(lengths, D, dt, D + len(lengths), rate=-5.0), dt, packed=packed)


@pytest.mark.parametrize("B,T,D,dtype,packed", [
    (3, 1200, 66, "bf16", False),   # 10 tiles a sequence forward
    (3, 640, 66, "bf16", False),    # 10 backward
    (3, 1920, 65, "f32", False),    # 16 and 30
    (5, 120, 64, "f32", False),     # one tile a sequence forward
    (5, 64, 130, "bf16", False),    # one backward
    (3, 960, 96, "bf16", True),     # 16 forward (60 tokens), 15 backward
    (4, 1920, 32, "f32", True),
])
def test_dense_sequences_of_whole_tiles(B, T, D, dtype, packed):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    log(f"glr dense {B} x {T} x {D} {dtype} packed={packed}")
    _check(_make([T] * B, D, dt, B + T + D, rate=-5.0), dt, packed=packed, dense=True)


@pytest.mark.parametrize("B,T,D,dtype,packed", [
    (4, 1920, 1408, "bf16", False),  # 64 x 11 forward, 120 x 11 backward
    (5, 1920, 513, "f32", False),    # 80 x 9, 150 x 9
    (4, 1920, 1280, "bf16", True),   # 128 x 5, 120 x 10
])
def test_dense_sequences_of_whole_tiles_several_a_workgroup(B, T, D, dtype, packed):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    log(f"glr dense {B} x {T} x {D} {dtype} packed={packed}")
    _check_wide(_make([T] * B, D, dt, B + T + D, rate=-5.0), dt, dense=True, packed=packed)
