"""The layer operators together, as a model uses them: convolution -> SiLU'd slices -> selective
scan for prompts; the same prompts token by token on slots; forks, clears and compaction of the
slots in between; and the convolution in front of the KDA operator, forward and backward."""

import numpy as np
import pytest
import torch

import gated_delta_rule_67_amd as kda
from oracle import conv, recurrent, selective_scan
from tests.helpers import assert_parity, log, to64

pytestmark = pytest.mark.gpu

H, G, K, V, W = 4, 2, 64, 32, 4
D = H * V + 2 * G * K


def _weights(seed):
    g = torch.Generator().manual_seed(seed)
    return dict(cw=0.5 * torch.randn(D, W, generator=g), cb=0.1 * torch.randn(D, generator=g),
                A_log=torch.log(1 + 3 * torch.rand(H, generator=g)), D=torch.randn(H, generator=g),
                dt_bias=0.5 * torch.randn(H, generator=g) - 1)


def _split(act):
    lead = act.shape[:-1]
    return (act[..., :H * V].unflatten(-1, (H, V)), act[..., H * V:H * V + G * K].unflatten(-1, (G, K)),
            act[..., H * V + G * K:].unflatten(-1, (G, K)))


def _prefill(w, proj, cu, conv0=None, ssm0=None):
    """proj [T, D + H]: a projection's output; its first D columns pass the convolution."""
    act, conv_state = kda.kda_conv_fwd(proj[:, :D], w["cw"], w["cb"], conv0, cu)
    x, b, c = _split(act)
    y, state = kda.kda_ssm_chunk_fwd(x, proj[:, D:], w["A_log"], b, c, w["D"], w["dt_bias"], ssm0, cu)
    return y, conv_state, state


def _step(w, proj, conv_pool, ssm_pool, slots):
    act = kda.kda_conv_step(proj[:, :D], w["cw"], conv_pool, w["cb"], slots)
    x, b, c = _split(act)
    return kda.kda_ssm_step(x, proj[:, D:], w["A_log"], b, c, ssm_pool, w["D"], w["dt_bias"], slots)


def test_prompts_then_tokens_on_forked_and_compacted_slots():
    w = {k: v.cuda() for k, v in _weights(0).items()}
    g = torch.Generator().manual_seed(1)
    lengths, more = [70, 5, 300], 6
    T = sum(lengths)
    proj = torch.randn(T, D + H, generator=g).to(torch.bfloat16).cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()
    y, cs, ss = _prefill(w, proj, cu)

    # the oracle of the prompts, on the activations that the convolution stored
    h = {k: to64(v) for k, v in w.items()}
    p64 = to64(proj)
    for n in range(3):
        a, b = int(cu[n]), int(cu[n + 1])
        act, _ = conv(p64[a:b, :D], h["cw"], h["cb"])
        act = to64(torch.from_numpy(act).to(torch.bfloat16))
        ry, rs, _, _ = selective_scan(act[:, :H * V].reshape(-1, H, V), p64[a:b, D:], h["A_log"],
                                      act[:, H * V:H * V + G * K].reshape(-1, G, K),
                                      act[:, H * V + G * K:].reshape(-1, G, K), h["D"], h["dt_bias"])
        assert_parity(to64(y[a:b]), ry, torch.bfloat16, f"y of prompt {n}", elem=False)
        assert_parity(to64(ss[n]), rs, torch.bfloat16, f"state of prompt {n}", elem=False)

    # slots: the prompts' states scattered over two pools, request 2 forked into slot 7
    conv_pool = torch.full((9, W - 1, D), float("nan"), dtype=torch.bfloat16).cuda()
    ssm_pool = torch.full((9, H, K, V), float("nan")).cuda()
    slots = torch.tensor([8, 3, 5], dtype=torch.int32).cuda()
    conv_pool[slots.long()], ssm_pool[slots.long()] = cs, ss
    pools = [conv_pool, ssm_pool]
    kda.kda_slots_copy(pools, torch.tensor([5, -1], dtype=torch.int32).cuda(), torch.tensor([7, 0], dtype=torch.int32).cuda())
    at = torch.tensor([8, 3, 5, 7, 0], dtype=torch.int32).cuda()  # the fork, and a new request on a cleared slot
    tokens = torch.randn(more, 5, D + H, generator=g).to(torch.bfloat16).cuda()
    tokens[:3, 3] = tokens[:3, 2]  # the fork goes the same way for three tokens
    out = [_step(w, t, conv_pool, ssm_pool, at) for t in tokens[:3]]
    assert all(torch.equal(o[2], o[3]) for o in out) and torch.equal(ssm_pool[5], ssm_pool[7])
    # compaction: five live slots move to the front, their requests' slots follow
    live = torch.zeros(9, dtype=torch.bool).cuda()
    live[at.long()] = True
    new, count = kda.kda_slots_compact(pools, live)
    at = new[at.long()].contiguous()
    assert int(count) == 5 and sorted(at.tolist()) == [0, 1, 2, 3, 4]
    out += [_step(w, t, conv_pool, ssm_pool, at) for t in tokens[3:]]
    out = torch.stack(out)

    # the same tokens as prompts continued from the states, and a fresh one
    cont = tokens.transpose(0, 1).reshape(5 * more, D + H).contiguous()
    cu5 = torch.arange(0, 5 * more + 1, more, dtype=torch.int32).cuda()
    y5, cs5, ss5 = _prefill(w, cont, cu5, torch.cat([cs, cs[2:], torch.zeros_like(cs[:1])]),
                            torch.cat([ss, ss[2:], torch.zeros_like(ss[:1])]))
    assert torch.equal(cs5, conv_pool[at.long()])
    assert_parity(to64(out.transpose(0, 1).reshape(5 * more, H, V)), to64(y5), torch.bfloat16, "steps against a prefill", elem=False)
    err = (ssm_pool[at.long()] - ss5).abs().max() / ss5.abs().max()
    log(f"    states of steps against a prefill: {float(err):.2e}")
    assert float(err) < 2.0 ** -15  # float32 sums of the same terms in another order


def test_convolution_in_front_of_kda_and_its_gradient():
    """q, k and v are slices of one convolved activation; the convolution's gradient from
    kda_chunk_bwd's dq, dk, dv, against central differences of the whole chain in float64."""
    B, T, HH, KK = 1, 64, 2, 32
    Dq = 3 * HH * KK
    g = torch.Generator().manual_seed(3)
    proj = torch.randn(B, T, Dq, generator=g).to(torch.bfloat16)
    cw, cb = 0.5 * torch.randn(Dq, W, generator=g), 0.1 * torch.randn(Dq, generator=g)
    gate = -0.1 * torch.rand(B, T, HH, KK, generator=g).to(torch.bfloat16)
    beta = torch.rand(B, T, HH, generator=g).to(torch.bfloat16)
    do = torch.randn(B, T, HH, KK, generator=g).to(torch.bfloat16)
    c = lambda t: t.cuda()  # noqa: E731
    act, _ = kda.kda_conv_fwd(c(proj), c(cw), c(cb))
    q, k, v = (t.reshape(B, T, HH, KK).contiguous() for t in act.split(HH * KK, dim=-1))
    flags = dict(qk_l2norm=True)
    o, _ = kda.kda_chunk_fwd(q, k, v, c(gate), c(beta), **flags)
    dq, dk, dv, _, _, _ = kda.kda_chunk_bwd(q, k, v, c(gate), c(beta), c(do), need_dh0=False, **flags)
    dact = torch.cat([t.flatten(2) for t in (dq, dk, dv)], dim=-1)
    dproj, dcw, dcb, _ = kda.kda_conv_bwd(c(proj), c(cw), dact, c(cb))

    def loss(p, w, b):
        a, _ = conv(p, w, b)
        a = a.reshape(1, T, 3, HH, KK)
        ref, _ = recurrent(torch.from_numpy(a[:, :, 0]), torch.from_numpy(a[:, :, 1]), torch.from_numpy(a[:, :, 2]),
                           gate, beta, 1.0 / np.sqrt(KK), None, qk_l2norm=True)
        return float((ref * to64(do)).sum())

    p64, w64, b64 = to64(proj)[0], to64(cw), to64(cb)
    r = np.random.default_rng(0)
    for name, got, arr in (("proj", to64(dproj)[0], 0), ("weight", to64(dcw), 1), ("bias", to64(dcb), 2)):
        args = [p64, w64, b64]
        worst, scale = 0.0, float(np.sqrt(np.mean(got ** 2)))
        for _ in range(12):
            i = tuple(r.integers(0, n) for n in args[arr].shape)
            up, down = args[arr].copy(), args[arr].copy()
            up[i] += 1e-5
            down[i] -= 1e-5
            diff = (loss(*[up if j == arr else a for j, a in enumerate(args)])
                    - loss(*[down if j == arr else a for j, a in enumerate(args)])) / 2e-5
            worst = max(worst, abs(diff - got[i]) / scale)
        log(f"    d{name}: worst |difference - gradient| / rms {worst:.3f}")
        # the activation and dq, dk, dv are rounded to bf16 on the way and the backward's own products
        # too: its tensors agree with the oracle's within 2e-2 of their rms a row (tests/helpers.py),
        # single elements within a few times that
        assert worst < 0.1
