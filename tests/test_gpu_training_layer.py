"""A layer of the norms, the recurrence and the checkpoints together, as training and serving use them:
norm in front (with the residual addition), projections, recurrence, norm behind under a gate and into
the residual. Gradients against float64 autograd of the same formulas on the CPU; prompts against
tokens one by one on a pool of states, with forks and compaction of its slots.

Tolerance in float32: an operator's outputs are within 1e-5 of their inputs' scale (each operator's own
tests bound it closer: about 100 roundings of 2^-24, 6e-6), a projection of 96 terms within 96 2^-24 = 6e-6,
and a gradient passes 6 operators and 4 projections, none of which enlarges a relative error by more than
its condition, under 10 here (sums of 96 terms of random signs): 10 stages x 1e-5 x 10 = 1e-3 of the
largest magnitude of the tensor."""

import numpy as np
import pytest
import torch

import gated_delta_rule_67_amd as kda
from tests.helpers import log

pytestmark = pytest.mark.gpu

D, F = 96, 96
LENGTHS = [130, 0, 1, 260]


def _params(seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    T = sum(LENGTHS)
    p = dict(x=r(T, D), res=r(T, D), w1=1 + 0.1 * r(D), s1=0.5 + 0.1 * r(D), proj=r(D, 4 * F) / D ** 0.5,
             A_log=0.3 * r(F) - 1, bias=r(F) - 1, w2=1 + 0.1 * r(F), s2=0.5 + 0.1 * r(F), init=r(len(LENGTHS), F))
    return p, r(T, F), r(len(LENGTHS), F)


def _reference(p, dout, dfinal):
    """Outputs and gradients in float64, by autograd."""
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    h = q["res"] + q["s1"] * q["x"]
    y = q["w1"] * h * torch.rsqrt(h.pow(2).mean(-1, keepdim=True) + 1e-6)
    x, r, i, z = (y @ q["proj"]).split(F, 1)
    g = -torch.exp(q["A_log"]) * torch.nn.functional.softplus(r + q["bias"])
    a, b = torch.exp(g), torch.sqrt(-torch.expm1(2 * g)) * torch.sigmoid(i) * x
    rows, finals, t = [], [], 0
    for n, m in enumerate(LENGTHS):
        s = q["init"][n]
        for _ in range(m):
            s = a[t] * s + b[t]
            rows.append(s)
            t += 1
        finals.append(s)
    o, final = torch.stack(rows), torch.stack(finals)
    out = h + q["s2"] * (q["w2"] * torch.sigmoid(z) * o * torch.rsqrt(o.pow(2).mean(-1, keepdim=True) + 1e-6))
    ((out * dout.double()).sum() + (final * dfinal.double()).sum()).backward()
    return out.detach(), {k: v.grad for k, v in q.items()}


def _cu():
    return torch.tensor(np.concatenate([[0], np.cumsum(LENGTHS)]), dtype=torch.int32, device="cuda")


def _layer(p, dout, dfinal, cu, packed=False):
    """Forward and backward through the library: (out, final state, gradients)."""
    y, h = kda.kda_prenorm_fwd(p["x"], p["w1"], p["res"], p["s1"])
    wide = y @ p["proj"]
    x, r, i, z = wide.split(F, 1)  # slices of one activation
    o, final, states = kda.kda_glr_fwd(x, r, p["A_log"], p["bias"], i, p["init"], cu, output_block_states=True)
    out = kda.kda_postnorm_fwd(o, p["w2"], z, h, p["s2"])
    keep = {"h": h, "x0": p["x"], "x": x, "r": r, "i": i, "z": z, "o": o}
    if packed:
        keep, states = {k: kda.kda_checkpoint_pack(v) for k, v in keep.items()}, None
    do, dz, dw2, ds2 = kda.kda_postnorm_bwd(keep["o"], p["w2"], dout, keep["z"], p["s2"])
    dx, dr, di, dA, db, dinit = kda.kda_glr_bwd(keep["x"], keep["r"], p["A_log"], do, p["bias"], keep["i"], p["init"], dfinal, cu,
                                                block_states=states)
    dwide = torch.cat([dx, dr, di, dz], 1)
    dres, dx0, dw1, ds1 = kda.kda_prenorm_bwd(keep["h"], p["w1"], dwide @ p["proj"].t(), dout, keep["x0"], p["s1"])
    return out, final, dict(x=dx0, res=dres, w1=dw1, s1=ds1, proj=y.t() @ dwide, A_log=dA, bias=db, w2=dw2, s2=ds2, init=dinit)


def test_gradients_of_a_layer():
    p, dout, dfinal = _params()
    ref, grads = _reference(p, dout, dfinal)
    dev = {k: v.cuda() for k, v in p.items()}
    out, _, got = _layer(dev, dout.cuda(), dfinal.cuda(), _cu())
    for name, a, b in [("out", out, ref)] + [(k, got[k], grads[k]) for k in grads]:
        err, top = float((a.double().cpu() - b).abs().max()), float(b.abs().max())
        log(f"    {name}: max |err| / max {err / top:.2e}")
        assert err <= 1e-3 * top, name


def test_training_step_from_checkpoints_in_a_graph():
    """The same step with everything kept in 8 bits, captured and replayed with changed inputs: each replay
    equals the eager call. A code is off by 2^-4 at most, so gradients are of the right size, not close."""
    p, dout, dfinal = _params(1)
    dev = {k: v.cuda() for k, v in p.items()}
    dout, dfinal, cu = dout.cuda(), dfinal.cuda(), _cu()
    exact = _layer(dev, dout, dfinal, cu)
    _layer(dev, dout, dfinal, cu, True)  # warms the projections' library up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, final, got = _layer(dev, dout, dfinal, cu, True)
    for k in range(3):
        dev["x"].mul_(-1)
        graph.replay()
        torch.cuda.synchronize()
        ref = _layer(dev, dout, dfinal, cu, True)
        assert torch.equal(out, ref[0]) and torch.equal(final, ref[1])
        for name in got:
            if name != "proj":  # a library product
                assert torch.equal(got[name], ref[2][name]), name
    dev["x"].mul_(-1)
    back = _layer(dev, dout, dfinal, cu, True)
    for name, a in exact[2].items():
        assert float((a - back[2][name]).norm()) <= 0.5 * float(a.norm()), name


def test_prompt_then_tokens_on_a_pool():
    """A prompt's final state goes into a slot, is forked, and both requests go on token by token; the pool
    is compacted in between. Outputs equal the prompt's own rows, to float32 rounding of the recurrence."""
    torch.manual_seed(3)
    T, cut, B = 90, 61, 5
    x, r, i = (torch.randn(1, T, F, device="cuda") for _ in range(3))
    A, bias, w = torch.randn(F, device="cuda") - 1, torch.randn(F, device="cuda"), torch.randn(F, device="cuda")
    y, final = kda.kda_glr_fwd(x, r, A, bias, i)
    _, s = kda.kda_glr_fwd(x[:, :cut], r[:, :cut], A, bias, i[:, :cut])
    pool = torch.full((B + 4, F), float("nan"), device="cuda")
    pool[6] = s[0]
    src, dst = torch.tensor([6], dtype=torch.int32, device="cuda"), torch.tensor([8], dtype=torch.int32, device="cuda")
    kda.kda_slots_copy(pool, src, dst)
    live = torch.zeros(B + 4, dtype=torch.bool, device="cuda")
    live[6] = live[8] = True
    new, count = kda.kda_slots_compact(pool, live)
    slots = torch.stack([new[6], torch.full_like(new[0], -1), new[8]])
    assert int(count) == 2
    for t in range(cut, T):
        row = lambda v: v[0, t].expand(3, F).contiguous()  # noqa: E731
        h = kda.kda_glr_step(row(x), row(r), A, pool, bias, row(i), slots)
        n = kda.kda_postnorm_fwd(h, w, row(i))
        assert torch.equal(h[0], h[2]) and not h[1].any() and torch.equal(n[0], n[2])
        # both sides within T (e_a + roundings) of the exact state: 90 tokens x about 60 2^-24, twice
        assert float((h[0] - y[0, t]).abs().max()) <= 2 * T * 60 * 2.0 ** -24 * max(1.0, float(y.abs().max()))
    assert float((pool[0] - final[0]).abs().max()) <= 2 * T * 60 * 2.0 ** -24 * max(1.0, float(y.abs().max()))
