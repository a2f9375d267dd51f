"""Cases that measure the short causal convolution, the selective state space scan and the
operations on slots of state pools: in plain torch operations and through the library.

``own`` False computes the operators in elementary torch operations (float32, sums and angles that
need it in float64); True calls the library. ``exact`` computes them in float64 token by token.
"""

import math
import random

import torch

own = False

_BF16, _F32 = torch.bfloat16, torch.float32


def listed():
    return [
        # q, k, v of a KDA layer (16 heads x 128) or x, B, C of a scan: a training / prefill batch
        dict(name="conv_fwd_b4_t8192_d6144", op="conv_fwd", dtype="bf16", seqs=4, tokens=32768,
             dim=6144, width=4, packed=False, init=False, silu=True),
        # a serving prefill of ragged prompts that continue cached ones, an odd channel count
        dict(name="conv_fwd_packed_t5003_d1030", op="conv_fwd", dtype="f32", seqs=23, tokens=5003,
             dim=1030, width=3, packed=True, init=True, silu=True),
        # the training batch of the first case, backward
        dict(name="conv_bwd_b4_t8192_d6144", op="conv_bwd", dtype="bf16", seqs=4, tokens=32768,
             dim=6144, width=4, packed=False, init=False, silu=True),
        # packed documents of one training row, gradients of the carried state included
        dict(name="conv_bwd_packed_t4097_d2048", op="conv_bwd", dtype="bf16", seqs=9, tokens=4097,
             dim=2048, width=4, packed=True, init=True, silu=True),
        # one interactive request: launch latency
        dict(name="conv_step_b1_d6144", op="conv_step", dtype="bf16", seqs=1, dim=6144, width=4,
             slots=8, silu=True),
        # a full decode batch against a pool of slots
        dict(name="conv_step_b256_d6144", op="conv_step", dtype="bf16", seqs=256, dim=6144, width=4,
             slots=320, silu=True),
        # a prefill batch of a scan layer with 64 heads x 64 and 8 groups of B, C
        dict(name="ssm_fwd_b4_t8192_h64", op="ssm_fwd", dtype="bf16", seqs=4, tokens=32768,
             heads=64, groups=8, state=128, head_dim=64, packed=False, init=False),
        # few heads, one long and several ragged prompts in one call, continued from cached states
        dict(name="ssm_fwd_packed_t16391_h16", op="ssm_fwd", dtype="bf16", seqs=5, tokens=16391,
             heads=16, groups=1, state=128, head_dim=128, packed=True, init=True),
        # a full decode batch
        dict(name="ssm_step_b256_h64", op="ssm_step", dtype="bf16", seqs=256, heads=64, groups=8,
             state=128, head_dim=64, slots=257),
        # one interactive request with few heads
        dict(name="ssm_step_b1_h16", op="ssm_step", dtype="bf16", seqs=1, heads=16, groups=1,
             state=128, head_dim=128, slots=4),
        # forks of shared prefixes and cleared slots over 18 layers' state pools
        dict(name="slots_copy_l18_s64_n24", op="slots_copy", dtype="f32", layers=18, slots=64,
             row=262144, pairs=24),
        # compaction of a half-empty pool of small states
        dict(name="slots_compact_l18_s96", op="slots_compact", dtype="bf16", layers=18, slots=96,
             row=18432, live=48),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "ssm_fwd", "ssm_fwd", "ssm_step",
                     "slots_copy", "slots_compact"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("conv_fwd", "conv_bwd"):
        tokens = _log_int(rng, 1, 32768)
        dim = _log_int(rng, 8, max(8, min(8192, 100_000_000 // tokens)))
        dim = dim if rng.random() < 0.3 else max(8, dim // 8 * 8)
        packed = rng.random() < 0.5
        seqs = _log_int(rng, 1, 64) if packed else rng.choice([n for n in (1, 2, 3, 4, 8) if tokens % n == 0])
        return dict(op=op, dtype=dtype, seqs=seqs, tokens=tokens, dim=dim, width=rng.choice([2, 3, 4, 4]),
                    packed=packed, init=rng.random() < 0.5, silu=rng.random() < 0.75)
    if op == "conv_step":
        seqs = _log_int(rng, 1, 512)
        dim = _log_int(rng, 64, 8192)
        dim = dim if rng.random() < 0.3 else dim // 8 * 8
        return dict(op=op, dtype=dtype, seqs=seqs, dim=dim, width=rng.choice([2, 3, 4, 4]),
                    slots=seqs + rng.randrange(0, 16), silu=rng.random() < 0.75)
    if op in ("ssm_fwd", "ssm_step"):
        groups = rng.choice([1, 1, 2, 4, 8])
        heads = groups * rng.choice([1, 2, 3, 4, 8])
        state = rng.choice([16, 32, 64, 64, 128, 128, 40, 33])
        head_dim = rng.choice([16, 32, 64, 64, 128, 48, 27])
        if op == "ssm_step":
            seqs = _log_int(rng, 1, 256)
            return dict(op=op, dtype=dtype, seqs=seqs, heads=heads, groups=groups, state=state,
                        head_dim=head_dim, slots=seqs + rng.randrange(0, 16))
        packed = rng.random() < 0.5
        tokens = _log_int(rng, 1, min(16384, 16_000_000_000 // (heads * state * head_dim)))
        seqs = _log_int(rng, 1, 8) if packed else rng.choice([n for n in (1, 2, 3, 4) if tokens % n == 0])
        return dict(op=op, dtype=dtype, seqs=seqs, tokens=tokens, heads=heads, groups=groups,
                    state=state, head_dim=head_dim, packed=packed, init=rng.random() < 0.5)
    slots = _log_int(rng, 4, 128)
    layers = _log_int(rng, 1, 24)
    row = _log_int(rng, 64, max(64, 1_000_000_000 // (4 * slots * layers)) if slots * layers > 900 else 262144)
    row = row if rng.random() < 0.3 else row // 8 * 8
    if op == "slots_copy":
        return dict(op=op, dtype=dtype, layers=layers, slots=slots, row=row, pairs=rng.randrange(1, slots // 2 + 1))
    return dict(op=op, dtype=dtype, layers=layers, slots=slots, row=row, live=rng.randrange(1, slots + 1))


# ---- inputs

def _lengths(case, seed):
    """Token counts of the sequences: equal ones, or ragged with empty and one-token sequences."""
    n, total = case["seqs"], case["tokens"]
    if not case["packed"]:
        return [total // n] * n
    r = random.Random(1000003 * seed + n)
    cuts = sorted(r.randrange(0, total + 1) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _cu(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def _dt_bias(u):
    """Biases whose softplus spreads over [1e-3, 1e-1] in its logarithm, as such layers start."""
    d = torch.exp(u * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
    return d + torch.log(-torch.expm1(-d))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=_F32):
        return torch.randn(shape, generator=gen, device="cuda", dtype=_F32).to(dtype)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device="cuda", dtype=_F32)

    op, dt = case["op"], _BF16 if case["dtype"] == "bf16" else _F32
    s = dict(case=case, op=op, dtype=dt)
    if op in ("conv_fwd", "conv_bwd"):
        lengths = _lengths(case, seed)
        t, d, w, n = case["tokens"], case["dim"], case["width"], case["seqs"]
        s.update(lengths=lengths, x=randn(t, d, dtype=dt), weight=randn(d, w) / math.sqrt(w), bias=0.1 * randn(d),
                 cu=_cu(lengths), initial=randn(n, w - 1, d, dtype=dt) if case["init"] else None)
        if op == "conv_bwd":
            s.update(dy=randn(t, d, dtype=dt), dfinal=randn(n, w - 1, d, dtype=dt) if case["init"] else None)
    elif op == "conv_step":
        n, d, w = case["seqs"], case["dim"], case["width"]
        s.update(x=randn(n, d, dtype=dt), weight=randn(d, w) / math.sqrt(w), bias=0.1 * randn(d),
                 pool=randn(case["slots"], w - 1, d, dtype=dt),
                 slots=torch.randperm(case["slots"], generator=gen, device="cuda")[:n].to(torch.int32))
    elif op in ("ssm_fwd", "ssm_step"):
        h, g, k, p, n = case["heads"], case["groups"], case["state"], case["head_dim"], case["seqs"]
        t = case["tokens"] if op == "ssm_fwd" else n
        # x, B and C are slices of one activation, as the convolution before them leaves it
        act = torch.nn.functional.silu(randn(t, h * p + 2 * g * k)).to(dt)
        s.update(x=act[:, :h * p].unflatten(1, (h, p)), b=act[:, h * p:h * p + g * k].unflatten(1, (g, k)),
                 c=act[:, h * p + g * k:].unflatten(1, (g, k)), dt=randn(t, h, dtype=dt),
                 A_log=torch.log(1 + 15 * rand(h)), D=1 + 0.1 * randn(h), dt_bias=_dt_bias(rand(h)))
        if op == "ssm_fwd":
            lengths = _lengths(case, seed)
            s.update(lengths=lengths, cu=_cu(lengths), initial=0.1 * randn(n, h, k, p) if case["init"] else None)
        else:
            s.update(pool=0.1 * randn(case["slots"], h, k, p),
                     slots=torch.randperm(case["slots"], generator=gen, device="cuda")[:n].to(torch.int32))
    else:
        n = case["slots"]
        s["pools"] = [randn(n, case["row"], dtype=dt) for _ in range(case["layers"])]
        perm = torch.randperm(n, generator=gen, device="cuda").to(torch.int32)
        if op == "slots_copy":
            # the first pairs' sources (some forked twice, some -1: clear) never are destinations
            m = case["pairs"]
            src = perm[m:][torch.randint(0, n - m, (m,), generator=gen, device="cuda")]
            s.update(src=torch.where(rand(m) < 0.2, torch.full_like(src, -1), src), dst=perm[:m].contiguous())
        else:
            live = torch.zeros(n, dtype=torch.bool, device="cuda")
            live[perm[:case["live"]].long()] = True
            s["live"] = live
    return s


# ---- the operators in elementary operations

def _positions(cu, tokens):
    """Of every token: its sequence, its place in it, the sequence's length."""
    t = torch.arange(tokens, device=cu.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t.to(torch.int32), right=True)
    start = cu.long()[seq]
    return seq, t - start, cu.long()[seq + 1] - start


def _rows(s, x):
    """The W - 1 rows before every sequence, then all tokens: the rows that taps read."""
    n, d, w = s["case"]["seqs"], s["case"]["dim"], s["case"]["width"]
    init = torch.zeros(n, w - 1, d, device=x.device) if s["initial"] is None else s["initial"].float()
    return torch.cat([init.reshape(n * (w - 1), d), x.float()])


def _tap_index(s):
    """[T, W]: the row of _rows that tap w of token t reads."""
    n, w = s["case"]["seqs"], s["case"]["width"]
    seq, pos, _ = _positions(s["cu"], s["case"]["tokens"])
    at = pos[:, None] + torch.arange(w, device=pos.device)  # place in (state ; sequence)
    return torch.where(at < w - 1, seq[:, None] * (w - 1) + at, n * (w - 1) + s["cu"].long()[seq][:, None] + at - (w - 1))


def _final_index(s):
    n, w = s["case"]["seqs"], s["case"]["width"]
    cu = s["cu"].long()
    at = (cu[1:] - cu[:-1])[:, None] + torch.arange(w - 1, device=cu.device)
    seq = torch.arange(n, device=cu.device)[:, None]
    return torch.where(at < w - 1, seq * (w - 1) + at, n * (w - 1) + cu[:-1, None] + at - (w - 1))


def _conv_fwd(s):
    rows = _rows(s, s["x"])
    pre = (rows[_tap_index(s)] * s["weight"].t()).sum(1) + s["bias"]
    y = pre * torch.sigmoid(pre) if s["case"]["silu"] else pre
    return y.to(s["dtype"]), rows[_final_index(s)].to(s["dtype"])


def _conv_bwd(s):
    case = s["case"]
    n, d, w, t = case["seqs"], case["dim"], case["width"], case["tokens"]
    rows, idx = _rows(s, s["x"]), _tap_index(s)
    taps = rows[idx]
    pre, dpre = (taps * s["weight"].t()).sum(1) + s["bias"], s["dy"].float()
    if case["silu"]:
        sg = torch.sigmoid(pre)
        dpre = dpre * (sg + pre * sg * (1 - sg))
    dweight, dbias = (dpre[:, None] * taps).sum(0).t().contiguous(), dpre.sum(0)
    # the row at place v of (state ; sequence) is tap k of the token at place v - k
    seq, pos, length = _positions(s["cu"], t)
    tap = torch.arange(w, device=pos.device)
    dpre = torch.cat([dpre, torch.zeros(1, d, device=dpre.device)])
    user = pos[:, None] + w - 1 - tap
    user = torch.where(user < length[:, None], s["cu"].long()[seq][:, None] + user, t)
    dx = (dpre[user] * s["weight"].t()).sum(1)
    cu = s["cu"].long()
    user = torch.arange(w - 1, device=pos.device)[:, None] - tap  # [W-1, W]
    user = torch.where((user >= 0) & (user < (cu[1:] - cu[:-1])[:, None, None]), cu[:-1, None, None] + user, t)
    dinit = (dpre[user] * s["weight"].t()).sum(2)
    if s["dfinal"] is not None:
        both = torch.cat([dinit.reshape(n * (w - 1), d), dx])
        both = both.index_add(0, _final_index(s).reshape(-1), s["dfinal"].float().reshape(-1, d))
        dinit, dx = both[:n * (w - 1)].reshape(n, w - 1, d), both[n * (w - 1):]
    out = [dx.to(s["dtype"]), dweight, dbias]
    return out + [dinit.to(s["dtype"])] if case["init"] else out


def _conv_step(s):
    at = s["slots"].long()
    rows = torch.cat([s["pool"][at], s["x"][:, None]], 1)
    pre = (rows.float() * s["weight"].t()).sum(1) + s["bias"]
    y = pre * torch.sigmoid(pre) if s["case"]["silu"] else pre
    s["pool"][at] = rows[:, 1:]
    return y.to(s["dtype"]), s["pool"]


def _softplus(z):
    return torch.clamp(z, min=0) + torch.log1p(torch.exp(-z.abs()))


def _padded(s):
    """[sequences, longest]: the token at every place, and whether there is one."""
    place = torch.arange(max(max(s["lengths"]), 1), device="cuda")
    cu = s["cu"].long()
    there = place < (cu[1:] - cu[:-1])[:, None]
    return torch.where(there, cu[:-1, None] + place, 0), there


_CHUNK = 64


def _ssm_fwd(s):
    """Chunks of 64 tokens: products inside a chunk, decayed sums of the chunks' states between."""
    case = s["case"]
    h, g, k, p, n = case["heads"], case["groups"], case["state"], case["head_dim"], case["seqs"]
    at, there = _padded(s)
    t = at.shape[1]
    nc = -(-t // _CHUNK)
    more = (0, nc * _CHUNK - t)
    at, there = torch.nn.functional.pad(at, more), torch.nn.functional.pad(there, more)

    def chunked(v):  # [T, heads, w] -> [n, nc, heads, 64, w], zeros where no token is
        v = torch.where(there[..., None, None], v[at].float(), 0.0)
        return v.reshape(n, nc, _CHUNK, v.shape[2], v.shape[3]).transpose(2, 3)

    x, b, c = chunked(s["x"]), chunked(s["b"]), chunked(s["c"])
    dt = torch.where(there[..., None], _softplus(s["dt"].float() + s["dt_bias"])[at], 0.0)
    dt = dt.reshape(n, nc, _CHUNK, h).transpose(2, 3)  # [n, nc, h, 64]
    total = (-torch.exp(s["A_log"].double())[:, None] * dt).cumsum(3)  # float64
    tri = torch.ones(_CHUNK, _CHUNK, dtype=torch.bool, device="cuda").tril()
    decay = torch.where(tri, total[..., :, None] - total[..., None, :], -math.inf).float().exp()
    scores = (c @ b.transpose(3, 4)).repeat_interleave(h // g, 2)
    y = (scores * decay * dt[..., None, :]) @ x
    weight = (total[..., -1:] - total).float().exp() * dt
    bh, ch = b.repeat_interleave(h // g, 2), c.repeat_interleave(h // g, 2)
    states = (bh * weight[..., None]).transpose(3, 4) @ x  # [n, nc, h, k, p]
    first = torch.zeros(n, 1, h, k, p, device="cuda") if s["initial"] is None else s["initial"][:, None]
    states = torch.cat([first, states], 1).transpose(1, 2).reshape(n, h, nc + 1, k * p)
    ends = torch.nn.functional.pad(total[..., -1].cumsum(1), (0, 0, 1, 0)).transpose(1, 2)  # [n, h, nc + 1]
    tri = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device="cuda").tril()
    between = torch.where(tri, ends[..., :, None] - ends[..., None, :], -math.inf).float().exp()
    entering = (between @ states).reshape(n, h, nc + 1, k, p).transpose(1, 2)
    y = y + (ch * total.float().exp()[..., None]) @ entering[:, :-1] + s["D"][:, None, None] * x
    y = y.transpose(2, 3).reshape(n, nc * _CHUNK, h, p)[there]
    return y.to(s["dtype"]), entering[:, -1].contiguous()


def _ssm_step(s):
    case = s["case"]
    at, r = s["slots"].long(), case["heads"] // case["groups"]
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    b, c = (s[m].float().repeat_interleave(r, 1) for m in ("b", "c"))
    x = s["x"].float()
    state = s["pool"][at] * torch.exp(-torch.exp(s["A_log"]) * dt)[..., None, None]
    state = state + b[..., :, None] * (dt[..., None] * x)[..., None, :]
    y = (state * c[..., None]).sum(2) + s["D"][:, None] * x
    s["pool"][at] = state
    return y.to(s["dtype"]), s["pool"]


def _slots_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for pool in s["pools"]:
        pool[dst] = torch.where(src[:, None] < 0, torch.zeros_like(pool[:1]), pool[src.clamp(min=0)])
    return s["pools"]


def _slots_compact(s):
    live = s["live"]
    n = live.sum()
    at = torch.arange(live.numel(), device="cuda")
    hole, mover = torch.nonzero(~live & (at < n))[:, 0], torch.nonzero(live & (at >= n))[:, 0]
    for pool in s["pools"]:
        pool[hole] = pool[mover]
    new = torch.where(live, at, -1)
    new[mover] = hole
    return s["pools"], new.to(torch.int32), n.to(torch.int32).reshape(1)


# ---- the same through the library

def _own(s):
    import gated_delta_rule_67_amd as kda

    case, op = s["case"], s["op"]
    if op in ("conv_fwd", "conv_bwd", "ssm_fwd"):
        cu = s["cu"] if case["packed"] else None

        def shaped(v):  # [T, ...] -> [B, T, ...] where the batch is dense
            return v if case["packed"] else v.unflatten(0, (case["seqs"], -1))

        if op == "conv_fwd":
            y, final = kda.kda_conv_fwd(shaped(s["x"]), s["weight"], s["bias"], s["initial"], cu, silu=case["silu"])
            return y.reshape(s["x"].shape), final
        if op == "conv_bwd":
            dx, dweight, dbias, dinit = kda.kda_conv_bwd(
                shaped(s["x"]), s["weight"], shaped(s["dy"]), s["bias"], s["initial"], s["dfinal"], cu,
                silu=case["silu"])
            out = [dx.reshape(s["x"].shape), dweight, dbias]
            return out + [dinit] if case["init"] else out
        y, final = kda.kda_ssm_chunk_fwd(shaped(s["x"]), shaped(s["dt"]), s["A_log"], shaped(s["b"]), shaped(s["c"]),
                                         s["D"], s["dt_bias"], s["initial"], cu)
        return y.reshape(s["x"].shape), final
    if op == "conv_step":
        return kda.kda_conv_step(s["x"], s["weight"], s["pool"], s["bias"], s["slots"], silu=case["silu"]), s["pool"]
    if op == "ssm_step":
        y = kda.kda_ssm_step(s["x"], s["dt"], s["A_log"], s["b"], s["c"], s["pool"], s["D"], s["dt_bias"], s["slots"])
        return y, s["pool"]
    if op == "slots_copy":
        kda.kda_slots_copy(s["pools"], s["src"], s["dst"])
        return s["pools"]
    new, count = kda.kda_slots_compact(s["pools"], s["live"])
    return s["pools"], new, count


_PLAIN = dict(conv_fwd=_conv_fwd, conv_bwd=_conv_bwd, conv_step=_conv_step, ssm_fwd=_ssm_fwd,
              ssm_step=_ssm_step, slots_copy=_slots_copy, slots_compact=_slots_compact)


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ---- what a pass cannot do without

def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("conv_fwd", "conv_bwd"):
        n = case["tokens"] * case["dim"]
        states = case["seqs"] * (case["width"] - 1) * case["dim"] * e
        if op == "conv_fwd":
            return dict(bytes=2 * e * n + states * (2 if case["init"] else 1), flops=(2 * case["width"] + 5) * n)
        return dict(bytes=3 * e * n + (3 * states if case["init"] else 0), flops=(6 * case["width"] + 10) * n)
    if op == "conv_step":
        n = case["seqs"] * case["dim"]
        return dict(bytes=2 * case["width"] * e * n + 4 * case["dim"] * (case["width"] + 1),
                    flops=(2 * case["width"] + 5) * n)
    if op in ("ssm_fwd", "ssm_step"):
        h, g, k, p, n = case["heads"], case["groups"], case["state"], case["head_dim"], case["seqs"]
        t = case["tokens"] if op == "ssm_fwd" else n
        states = 4 * n * h * k * p * (2 if op == "ssm_step" or case["init"] else 1)
        return dict(bytes=t * e * (2 * h * p + 2 * g * k + h) + states, flops=4 * t * h * k * p)
    size = e * case["layers"] * case["row"]
    # of a compaction: the live slots that lie behind the first `live` ones, on average
    moved = case["pairs"] if op == "slots_copy" else case["live"] * (case["slots"] - case["live"]) / case["slots"]
    return dict(bytes=2 * moved * size + 8 * case["slots"], flops=0)


# ---- the definitions in float64

def _conv_exact(s):
    case = s["case"]
    w, d, n = case["width"], case["dim"], case["seqs"]
    x, weight, bias = s["x"].double(), s["weight"].double(), s["bias"].double()
    init = torch.zeros(n, w - 1, d, dtype=torch.float64, device="cuda") if s["initial"] is None else s["initial"].double()
    bwd = case["op"] == "conv_bwd"
    if bwd:
        dy = s["dy"].double()
        dfinal = torch.zeros_like(init) if s["dfinal"] is None else s["dfinal"].double()
    ys, finals, dxs, dinits = [], [], [], []
    dweight, dbias = torch.zeros_like(weight), torch.zeros_like(bias)
    at = 0
    for i, m in enumerate(s["lengths"]):
        full = torch.cat([init[i], x[at:at + m]])
        pre = bias + sum(weight[:, j] * full[j:j + m] for j in range(w))
        sg = torch.sigmoid(pre)
        ys.append(pre * sg if case["silu"] else pre)
        finals.append(full[m:])
        if bwd:
            dpre = dy[at:at + m] * ((sg + pre * sg * (1 - sg)) if case["silu"] else 1.0)
            dfull = torch.zeros_like(full)
            dfull[m:] += dfinal[i]
            for j in range(w):
                dfull[j:j + m] += weight[:, j] * dpre
                dweight[:, j] += (dpre * full[j:j + m]).sum(0)
            dbias += dpre.sum(0)
            dxs.append(dfull[w - 1:])
            dinits.append(dfull[:w - 1])
        at += m
    if bwd:
        out = [torch.cat(dxs), dweight, dbias]
        return out + [torch.stack(dinits)] if case["init"] else out
    return torch.cat(ys), torch.stack(finals)


def _ssm_token(state, x, dt, a, b, c, skip):
    """One token: the state [n, h, k, p] after it and its output."""
    state = state * torch.exp(a * dt)[..., None, None] + b[..., :, None] * (dt[..., None] * x)[..., None, :]
    return state, (state * c[..., None]).sum(2) + skip[:, None] * x


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("slots_copy", "slots_compact"):
        return None  # copies: no computed numbers
    if op in ("conv_fwd", "conv_bwd"):
        return _conv_exact(s)
    if op == "conv_step":
        at = s["slots"].long()
        rows = torch.cat([s["pool"][at], s["x"][:, None]], 1).double()
        pre = (rows * s["weight"].double().t()).sum(1) + s["bias"].double()
        pool = s["pool"].double()
        pool[at] = rows[:, 1:]
        return (pre * torch.sigmoid(pre) if case["silu"] else pre), pool
    r = case["heads"] // case["groups"]
    dt = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=1000.0)
    a, skip, x = -torch.exp(s["A_log"].double()), s["D"].double(), s["x"]
    if op == "ssm_step":
        at = s["slots"].long()
        b, c = (s[m].double().repeat_interleave(r, 1) for m in ("b", "c"))
        pool = s["pool"].double()
        pool[at], y = _ssm_token(pool[at], x.double(), dt, a, b, c, skip)
        return y, pool
    n, h, k, p = case["seqs"], case["heads"], case["state"], case["head_dim"]
    state = torch.zeros(n, h, k, p, dtype=torch.float64, device="cuda") if s["initial"] is None else s["initial"].double()
    y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    # the sequences side by side, longest first, so that those which have ended drop off the end
    order = sorted(range(n), key=lambda i: -s["lengths"][i])
    lengths = [s["lengths"][i] for i in order]
    starts = [sum(s["lengths"][:i]) for i in order]
    pick = torch.tensor(order, device="cuda")
    state, first = state[pick], torch.tensor(starts, device="cuda")
    for t in range(lengths[0]):
        m = sum(1 for v in lengths if v > t)
        at = first[:m] + t
        b, c = (s[v][at].double().repeat_interleave(r, 1) for v in ("b", "c"))
        state[:m], y[at] = _ssm_token(state[:m], x[at].double(), dt[at], a, b, c, skip)
    final = torch.empty_like(state)
    final[pick] = state
    return y, final
