"""What is measured of attention on (C, e) tensors: over whole prompts with its gradient, rotary positions, and the form
that answers single tokens from a cache of 4-bit mantissas.

Every tensor is a pair of int8 mantissas C and int8 exponents e, value C * 2^e; an output comes back as both, whole
numbers that have to be equal bit for bit.  Q, K and V are the columns of one matrix [tokens x (heads + 2 kv_heads) *
head_dim], as the projection in front of them writes it, one exponent per token or one for all.

The arithmetic is the library's contract.  Products and sums are exact integers.  A softmax weight is 2^x at a resolution
of 2^-17 in x, from a polynomial in fp32, and enters the sums as an integer of at most 32512 (in the key's gradient, whose
rows differ most, of at most 64 times that); so the sums are exact in any order.  Results are rounded into their groups once, from 53 bits.  The plain form below computes that with elementary
torch operations over sequences padded to one length, in 32 bits where the definition says so and else in 64.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
E_LO, E_HI = -48, 16             # exponents of Q, K, V and O are read clipped to these
UNIT = 32512                     # a weight of one
POLY = (2545.0, 7358.0, 22609.0, 32512.0)  # 32512 * 2^f on [0, 1), highest power first
BLOCK = 256                      # keys of a cache that share one maximum


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one step of a server answering 16 sequences, rotated before it enters the cache: latency
        dict(name="rope_step_16x48x128", op="rope", rows=16, heads=32, kv_heads=8, head_dim=128, rot=128,
             interleaved=False, inverse=False, group="row", scaling="parts", far=40000),
        # the gradient through the rotation of half of every head, a ViT-B batch of tokens
        dict(name="rope_back_25216x36x64", op="rope", rows=25216, heads=12, kv_heads=12, head_dim=64, rot=32,
             interleaved=True, inverse=True, group="row", scaling="none", far=197),
        # the smallest configuration: latency
        dict(name="attn_1x64_4h32", op="attn_fwd", n=1, rows=64, spread="even", spare=0, heads=4, kv_heads=4,
             head_dim=32, causal=True, group="tensor", stats=False),
        # every image of a ViT-B batch of 128, 197 tokens each, all of which see each other
        dict(name="attn_128x197_12h64", op="attn_fwd", n=128, rows=25216, spread="even", spare=0, heads=12, kv_heads=12,
             head_dim=64, causal=False, group="row", stats=True),
        # prompts of different lengths packed behind each other, grouped heads, padding rows at the end
        dict(name="attn_5x8192_32h128", op="attn_fwd", n=5, rows=8192, spread="ragged", spare=37, heads=32, kv_heads=8,
             head_dim=128, causal=True, group="row", stats=False),
        # the gradient of the ViT-B batch
        dict(name="attn_bwd_128x197_12h64", op="attn_bwd", n=128, rows=25216, spread="even", spare=0, heads=12,
             kv_heads=12, head_dim=64, causal=False, group="row"),
        # the gradient over packed causal sequences with grouped heads
        dict(name="attn_bwd_3x4096_16h64", op="attn_bwd", n=3, rows=4096, spread="ragged", spare=5, heads=16, kv_heads=4,
             head_dim=64, causal=True, group="row"),
        # the new tokens of 16 sequences enter the cache: latency
        dict(name="store_16_8h128", op="store", rows=16, heads=32, kv_heads=8, head_dim=128, page=16, group="row"),
        # a prompt enters the cache
        dict(name="store_8192_8h128", op="store", rows=8192, heads=32, kv_heads=8, head_dim=128, page=64, group="row"),
        # one short sequence answered: latency
        dict(name="cache_1x300_8h64", op="cache", n=1, longest=300, spread="even", heads=8, kv_heads=8, head_dim=64,
             page=16, group="row"),
        # a batch of sequences of different lengths
        dict(name="cache_48x8000_32h128", op="cache", n=48, longest=8000, spread="ragged", heads=32, kv_heads=8,
             head_dim=128, page=64, group="row"),
        # one long context
        dict(name="cache_1x131072_32h128", op="cache", n=1, longest=131072, spread="even", heads=32, kv_heads=8,
             head_dim=128, page=256, group="row"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "store", "cache", "cache"])
    group = rng.choice(["row", "row", "tensor"])
    heads, kv_heads = rng.choice([(1, 1), (3, 3), (12, 12), (8, 2), (16, 4), (32, 8), (6, 2), (10, 1)])
    if op == "rope":
        head_dim = rng.choice([32, 40, 64, 80, 128])
        width = (heads + 2 * kv_heads) * head_dim
        return dict(op=op, rows=_log(rng, 1, max(2, 56_000_000 // width)), heads=heads, kv_heads=kv_heads,
                    head_dim=head_dim, rot=rng.choice([head_dim, head_dim, head_dim // 2]),
                    interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5, group=group,
                    scaling=rng.choice(["none", "linear", "parts"]), far=_log(rng, 1, 40000))
    if op in ("attn_fwd", "attn_bwd"):
        head_dim, causal = rng.choice([32, 40, 64, 64, 80, 128]), rng.random() < 0.5
        most = 1.2e8 if op == "attn_fwd" else 5e7
        while True:
            n, mean = _log(rng, 1, 128), _log(rng, 1, 4096)
            spread = rng.choice(["even", "ragged"])
            c = dict(op=op, n=n, rows=n * mean, spread=spread, spare=rng.choice([0, 0, 7]), heads=heads,
                     kv_heads=kv_heads, head_dim=head_dim, causal=causal, group=group)
            tall = max(_lengths(c))
            if n * tall * tall * heads * head_dim <= 64 * most and n * tall * heads * head_dim <= 2e7:
                break
        if op == "attn_fwd":
            c["stats"] = rng.random() < 0.5
        return c
    head_dim = rng.choice([32, 64, 96, 128])
    page = rng.choice([1, 16, 32, 64, 128, 256])
    if op == "store":
        return dict(op=op, rows=_log(rng, 1, 8192), heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page,
                    group=group)
    while True:
        n, longest = _log(rng, 1, 128), _log(rng, 1, 131072)
        if n * longest * kv_heads * head_dim <= 1e8 and n * longest * heads <= 4e6:
            return dict(op=op, n=n, longest=longest, spread=rng.choice(["even", "ragged"]), heads=heads,
                        kv_heads=kv_heads, head_dim=head_dim, page=page, group=group)


def _lengths(case):
    """How many tokens each sequence of a case has: the same for every seed, the first one the longest."""
    n = case["n"]
    if case["op"] == "cache":
        rng = random.Random(case["longest"] * 131 + n)
        if case["spread"] == "even":
            return [case["longest"]] * n
        return [case["longest"]] + [rng.randint(0, case["longest"]) for _ in range(n - 1)]
    rows = max(case["rows"] - case["spare"], n)
    if case["spread"] == "even":
        return [rows // n] * n
    rng = random.Random(rows * 131 + n)
    parts = [rng.expovariate(1.0) for _ in range(n)]
    got = [max(1, int(rows * p / sum(parts))) for p in parts]
    while sum(got) > rows:
        got[got.index(max(got))] -= 1
    return sorted(got, reverse=True)


def _rows(case):
    return max(case["rows"], sum(_lengths(case)) + case["spare"])


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _tokens(g, rows, cols, group, scale=1.0):
    """Activations or gradients whose rows differ in size, as a network's do: each group's largest magnitude is 127."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x = x * (scale * torch.exp2(0.7 * torch.randn(rows, 1, generator=g, device=DEV)))
    mx = x.abs().amax(dim=1, keepdim=True) if group == "row" else x.abs().max().reshape(1, 1)
    mx = mx.clamp_min(1e-30)
    c = torch.round(x * (127.0 / mx)).to(torch.int8)
    e = (torch.ceil(torch.log2(mx)) - 7).to(torch.int8).reshape(-1)
    return c.contiguous(), e.contiguous()


def _frequencies(case):
    """Turns of a token's angle by dimension pair, stretched for contexts longer than the trained ones."""
    rot, base = case["rot"], 10000.0
    factor, trained = {"none": (1.0, 0.0), "linear": (4.0, 0.0), "parts": (8.0, 8192.0)}[case["scaling"]]
    out = []
    for k in range(rot // 2):
        w = math.pow(base, -2.0 * k / rot)
        if trained > 0.0:
            keep = min(max((trained * w / (2.0 * math.pi) - 1.0) / (4.0 - 1.0), 0.0), 1.0)
        else:
            keep = 0.0
        out.append(w * (keep + (1.0 - keep) / factor))
    return out, dict(base=base, factor=factor, trained=trained, low=1.0, high=4.0)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, group = case["op"], case["group"]
    width = (case["heads"] + 2 * case["kv_heads"]) * case["head_dim"]
    s = dict(case=case)
    if op == "rope":
        s["x"] = _tokens(g, case["rows"], width, group)
        s["pos"] = torch.randint(0, case["far"], (case["rows"],), generator=g, device=DEV, dtype=torch.int32)
        angle = torch.arange(case["far"], device=DEV).double().reshape(-1, 1) * torch.tensor(
            _frequencies(case)[0], device=DEV, dtype=torch.float64)
        turn = torch.stack([torch.cos(angle), torch.sin(angle)], 2)
        s["table"] = torch.round(turn * 2.0 ** 14).to(torch.int16)
    elif op in ("attn_fwd", "attn_bwd"):
        lengths = _lengths(case)
        s["x"] = _tokens(g, _rows(case), width, group, scale=0.7)
        at = np.concatenate([[0], np.cumsum(lengths)])
        s["offsets"] = torch.from_numpy(at.astype(np.int32)).to(DEV)
        tall = max(lengths)
        idx = torch.from_numpy(np.minimum(at[:-1, None] + np.arange(tall)[None], _rows(case) - 1)).to(DEV)
        s["index"] = idx  # the padded form's gather, [n x longest]
        s["live"] = torch.arange(tall, device=DEV)[None] < torch.tensor(lengths, device=DEV)[:, None]
        s["scale"] = float(np.float32(case["head_dim"] ** -0.5))
        if op == "attn_bwd":
            s["dy"] = _tokens(g, _rows(case), case["heads"] * case["head_dim"], group, scale=2.0 ** -10)
            got = _attn_fwd(dict(case, stats=True), s)
            s["o"], s["stats"] = (got["mant"], got["exp"]), got["stats"]
    else:
        kv, d, page = case["kv_heads"], case["head_dim"], case["page"]
        if op == "store":
            rows, per = case["rows"], None
            pages = -(-rows // page) + 3
            s["x"] = _tokens(g, rows, width, group)
            s["slots"] = torch.randperm(pages * page, generator=g, device=DEV)[:rows].to(torch.int32)
            s["slots"][rows // 2::97] = -1  # rows of padding are not stored
        else:
            lengths = _lengths(case)
            per = max(1, -(-max(lengths) // page))
            pages = sum(-(-t // page) for t in lengths) + 3
            s["x"] = _tokens(g, case["n"], width, group, scale=0.7)
            order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
            table, used = np.full((case["n"], per), -1, np.int64), 0
            for i, t in enumerate(lengths):
                k = -(-t // page)
                table[i, :k] = np.arange(used, used + k)
                used += k
            at = torch.from_numpy(table).to(DEV)
            s["pages"] = torch.where(at >= 0, order[at.clamp_min(0)], -1).to(torch.int32)
            s["lengths"] = torch.tensor(lengths, device=DEV, dtype=torch.int32)
            s["scale"] = float(np.float32(d ** -0.5))
        for name, spread in (("k", 2.2), ("v", 2.2)):
            x = torch.empty(pages, page, kv, d, device=DEV)
            x.normal_(generator=g)
            c = torch.round(x * spread).clamp(-7, 7).to(torch.int32) & 15
            s[name] = (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8).contiguous()
            s[name + "e"] = torch.randint(-4, 0, (pages, page, kv), generator=g, device=DEV, dtype=torch.int32).to(torch.int8)
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program that uses the library keeps: tensors as (C, e) matrices, outputs, a workspace, a table of angles."""
    from integer_only_dnn_amd import ie
    case = s["case"]
    op, heads, kv, d = case["op"], case["heads"], case["kv_heads"], case["head_dim"]

    def mat(t):
        return ie.Mat(t[0], t[1], ie.TENSOR if case["group"] == "tensor" else ie.ROW)

    h = dict(ws=ie.Workspace(DEV), x=mat(s["x"]))
    rows, width = s["x"][0].shape
    if op == "rope":
        h["rope"] = ie.Rope(d, case["rot"], case["far"], interleaved=case["interleaved"], device=DEV,
                            **_frequencies(case)[1])
        h["y"] = ie.Mat.empty(rows, width, ie.TENSOR if case["group"] == "tensor" else ie.ROW, DEV)
    elif op in ("attn_fwd", "attn_bwd"):
        h["plan"] = ie.Attention(heads, kv, d, s["scale"], case["causal"], s["offsets"])
        if op == "attn_fwd":
            # rows behind the last sequence are not written: they start as what the plain form has there
            h["o"] = ie.Mat(torch.zeros(rows, heads * d, dtype=torch.int8, device=DEV),
                            torch.full((rows,), -128, dtype=torch.int8, device=DEV), ie.ROW)
            h["stats"] = torch.zeros(rows, heads, 2, dtype=torch.int32, device=DEV) if case["stats"] else None
        else:
            h["o"], h["dy"] = ie.Mat(*s["o"], ie.ROW), mat(s["dy"])
            h["dx"] = ie.Mat(torch.zeros(rows, width, dtype=torch.int8, device=DEV),
                             torch.full((rows,), -128, dtype=torch.int8, device=DEV), ie.ROW)
    else:
        h["cache"] = ie.Cache(s["k"], s["ke"], s["v"], s["ve"])
        if op == "cache":
            h["plan"] = ie.Attention(heads, kv, d, s["scale"])
            h["o"] = ie.Mat.empty(rows, heads * d, ie.ROW, DEV)
    s["h"] = h


# --------------------------------------------------------------------------
# The plain form
# --------------------------------------------------------------------------

def _exp2(e):
    """2^e in float64, exactly (e a whole number within the normal range)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _clip(e):
    return e.to(torch.int64).clamp(E_LO, E_HI)


def _per_row(t):
    """The exponent of every row, [rows], of a matrix with one per row or one in all."""
    c, e = t
    return e.to(torch.int64).expand(c.shape[0]) if e.numel() == 1 else e.to(torch.int64)


def _round(y, group, most=127):
    """Values into groups along the last axis: the smallest exponent that holds the largest magnitude, ties to even."""
    mx = y.abs().amax(dim=-1, keepdim=True) if group == "row" else y.abs().max().reshape([1] * y.dim())
    _, x = torch.frexp(mx)
    e = x.to(torch.int64) - (7 if most == 127 else 3)
    e = torch.where(torch.round(mx * _exp2(-e)) > most, e + 1, e)
    e = torch.where(mx == 0, torch.full_like(e, -128), e).clamp_min(-128)
    return torch.round(y * _exp2(-e)).to(torch.int8), e.to(torch.int8)


def _weight(d, r):
    """32512 * 2^(d r) for d <= 0, both float32: the exponent at a resolution of 2^-17 and at least -32, the power of its
    fraction from a polynomial in float32 (each step one rounding, as products and sums of a step are exact in 64 bits)."""
    y = torch.round((d.double() * r.double()).clamp_min(-64.0) * 2.0 ** 17).mul_(2.0 ** -17).clamp_min_(-32.0)
    n = torch.floor(y)
    f = y - n
    q = (f * POLY[0] + POLY[1]).float().double()
    q = (q * f + POLY[2]).float().double()
    q = (q * f + POLY[3]).float().double()
    return (q * _exp2(n)).float()


def _rope(case, s):
    (c, _), d, rot = s["x"], case["head_dim"], case["rot"]
    rows, k = c.shape[0], case["heads"] + case["kv_heads"]
    x = c.reshape(rows, -1, d).double()
    cos, sin = s["table"][s["pos"].long()].double().reshape(rows, 1, -1, 2).unbind(3)
    if case["inverse"]:
        sin = -sin
    y = x * 2.0 ** 14
    if case["interleaved"]:
        a, b = x[:, :k, 0:rot:2], x[:, :k, 1:rot:2]
        y[:, :k, 0:rot:2], y[:, :k, 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[:, :k, :rot // 2], x[:, :k, rot // 2:rot]
        y[:, :k, :rot // 2], y[:, :k, rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    y = y.reshape(rows, -1) * _exp2(_per_row(s["x"]) - 14).reshape(-1, 1)
    mant, exp = _round(y, case["group"])
    return dict(mant=mant, exp=exp.reshape(-1))


def _padded(case, s):
    """Q, K, V as [n, kv_heads, queries or keys, head_dim] (a group's query heads behind each other), float32."""
    h, kv, d = case["heads"], case["kv_heads"], case["head_dim"]
    n, tall = s["index"].shape
    x = s["x"][0][s["index"]].float().reshape(n, tall, h + 2 * kv, d)
    x = x * s["live"][:, :, None, None]
    q = _stack(x[:, :, :h], kv)
    return q, x[:, :, h:h + kv].transpose(1, 2).contiguous(), x[:, :, h + kv:].transpose(1, 2).contiguous()


def _stack(x, kv):
    """[n, tall, heads, d] as [n, kv_heads, group * tall, d]."""
    n, tall, h, d = x.shape
    return x.reshape(n, tall, kv, h // kv, d).permute(0, 2, 3, 1, 4).reshape(n, kv, h // kv * tall, d).contiguous()


def _unstack(x, case):
    """[n, kv_heads, group * tall, d] as [n, tall, heads * d]."""
    n, kv, _, d = x.shape
    g = case["heads"] // kv
    return x.reshape(n, kv, g, -1, d).permute(0, 3, 1, 2, 4).reshape(n, -1, kv * g * d)


def _seen(case, s):
    """Which keys a query sees, [n, 1, group * tall, tall], and their exponents (clipped), [n, tall]."""
    n, tall = s["index"].shape
    see = s["live"][:, None, :] & s["live"][:, :, None]
    if case["causal"]:
        see = see & torch.ones(tall, tall, dtype=torch.bool, device=DEV).tril()[None]
    g = case["heads"] // case["kv_heads"]
    e = torch.where(s["live"], _clip(_per_row(s["x"]))[s["index"]], E_LO)
    return see[:, None].repeat(1, 1, g, 1), e


def _rates(case, s, e):
    """2^(score) per unit of a query's products: float32 [n, 1, group * tall, 1]."""
    c = torch.tensor(s["scale"] * math.log2(math.e), device=DEV, dtype=torch.float64).float()
    r = (c.double() * _exp2(e)).float()
    return r.repeat(1, case["heads"] // case["kv_heads"])[:, None, :, None]


def _put(case, s, y, width):
    """Values of the padded rows, [n, tall, width], rounded by row, in the packed rows they belong to."""
    mant = torch.zeros(_rows(case), width, dtype=torch.int8, device=DEV)
    exp = torch.full((_rows(case),), -128, dtype=torch.int8, device=DEV)
    c, e = _round(y, "row")
    at = s["index"][s["live"]]
    mant[at], exp[at] = c[s["live"]], e[..., 0][s["live"]]
    return dict(mant=mant, exp=exp)


def _attn_fwd(case, s):
    q, k, v = _padded(case, s)
    see, e = _seen(case, s)
    f = _exp2(e)[:, None, None, :]
    t = (q @ k.transpose(2, 3).contiguous()) * f.float()
    t = torch.where(see, t, -math.inf)
    m = t.amax(dim=3, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    w = torch.where(see, _weight((t - m).clamp_min(-3e38), _rates(case, s, e)), 0.0).double()
    total = torch.round(w).sum(dim=3, keepdim=True)
    top = e.cummax(dim=1).values if case["causal"] else e.amax(dim=1, keepdim=True).expand_as(e)
    top = top.repeat(1, case["heads"] // case["kv_heads"])[:, None, :, None]
    p = torch.round(w * (f * _exp2(-top)))
    y = (p @ v.double()) * (1.0 / total.clamp_min(1.0)) * _exp2(top)
    out = _put(case, s, _unstack(y, case), case["heads"] * case["head_dim"])
    if case["stats"]:
        pair = torch.cat([m.view(torch.int32), total.to(torch.int32)], 3)
        stats = torch.zeros(_rows(case), case["heads"], 2, dtype=torch.int32, device=DEV)
        stats[s["index"][s["live"]]] = _unstack(pair, case).reshape(*s["index"].shape, -1, 2)[s["live"]]
        out["stats"] = stats
    return out


def _bits(n):
    """Bits of a whole number >= 0 (float64): the smallest b with n < 2^b."""
    return torch.frexp(n)[1].to(torch.int64)


def _later(x, case):
    """The largest value over the queries that see a key: [n, kv_heads, group, tall] to [n, kv_heads, tall]."""
    x = x.amax(dim=2)
    if not case["causal"]:
        return x.amax(dim=2, keepdim=True).expand_as(x)
    return x.flip(2).cummax(dim=2).values.flip(2)


def _attn_bwd(case, s):
    h, kv, d = case["heads"], case["kv_heads"], case["head_dim"]
    g = h // kv
    n, tall = s["index"].shape
    q, k, v = _padded(case, s)
    see, e = _seen(case, s)
    f = _exp2(e)[:, None, None, :]
    live = s["live"][:, None, None, :]
    dy = _stack(s["dy"][0][s["index"]].float().reshape(n, tall, h, d) * s["live"][:, :, None, None], kv)
    o = _stack(s["o"][0][s["index"]].float().reshape(n, tall, h, d) * s["live"][:, :, None, None], kv)
    m, total = _stack(s["stats"][s["index"]], kv).split(1, dim=3)
    m, total = m.view(torch.float32), total.to(torch.int64) & 0xFFFFFFFF
    m, total = (torch.where(s["live"].repeat(1, g)[:, None, :, None], x, 1) for x in (m, total))
    eo = torch.where(s["live"], _clip(_per_row(s["o"]))[s["index"]], E_LO).repeat(1, g)[:, None, :, None]
    ed = torch.where(s["live"], _per_row(s["dy"])[s["index"]], -128)
    most = ed.amax(dim=1, keepdim=True)

    # weights, and what a weight's gradient is in units of its row's gradient exponent
    t = (q @ k.transpose(2, 3).contiguous()) * f.float()
    w = torch.where(see, _weight((t - m).clamp_max(0.0), _rates(case, s, e)), 0.0)
    dot = (dy.double() * o.double()).sum(dim=3, keepdim=True)
    u = (dy @ v.transpose(2, 3).contiguous()) * f.float() - (dot * _exp2(eo)).float()
    su = w * u

    # powers of two that bound them
    beta = (_bits((dy.double() ** 2).sum(dim=3)) + 1).div(2, rounding_mode="floor").reshape(n, kv, g, tall)
    delta = (_bits(dot.abs()) + eo).reshape(n, kv, g, tall)
    nu = (_bits((v.double() ** 2).sum(dim=3)) + 1).div(2, rounding_mode="floor") + e[:, None, :]
    nu = torch.where(live[:, 0], nu, -1000)
    high, both = nu.amax(dim=2)[:, :, None, None], (nu + e[:, None, :]).amax(dim=2)[:, :, None, None]
    sigma = torch.maximum(beta + both, delta + e.amax(dim=1)[:, None, None, None]) + 1
    sigma = sigma.reshape(n, kv, g * tall, 1)
    b = torch.round((su * f.float()).double() * _exp2(-sigma))
    rate = s["scale"] / total.double()
    dq = (b @ k.double()) * rate * _exp2(sigma + ed.repeat(1, g)[:, None, :, None])

    a = (1.0 / total.double()).float().double() * _exp2((ed - most).clamp_min(-60)).repeat(1, g)[:, None, :, None]
    alpha = torch.where(live, _bits(a).reshape(n, kv, g, tall), -1000)
    kappa = _later(alpha, case)[:, :, None, :]
    av = torch.round((w * a.float()).double() * _exp2(-kappa.clamp_min(-900)))
    av = torch.where(see, av, 0.0)
    dv = (av.transpose(2, 3).contiguous() @ dy.double()) * _exp2(kappa.clamp_min(-900).transpose(2, 3) + most[:, :, None, None])

    eq = e[:, None, None, :]
    lam = torch.maximum(_later(alpha + eq + beta, case) + high[:, :, 0], _later(alpha + eq + delta, case)) + 1
    lam = torch.where(live[:, 0], lam, -1000)
    whole = lam.amax(dim=2)[:, :, None]
    lam = (lam - whole).clamp_min(-96)[:, :, None, :]
    bi = (a * _exp2(e.repeat(1, g)[:, None, :, None] - whole[..., None])).float()
    cv = torch.where(see, torch.round((su * bi).double() * _exp2(6 - lam)), 0.0)
    dk = (cv.transpose(2, 3).contiguous() @ q.double()) * s["scale"] * _exp2(
        lam.transpose(2, 3) - 6 + whole[..., None] + most[:, :, None, None])

    y = torch.cat([_unstack(dq, case), dk.transpose(1, 2).reshape(n, tall, -1), dv.transpose(1, 2).reshape(n, tall, -1)], 2)
    return _put(case, s, y, (h + 2 * kv) * d)


def _store(case, s):
    h, kv, d = case["heads"], case["kv_heads"], case["head_dim"]
    c = s["x"][0].reshape(-1, h + 2 * kv, d)
    value = c[:, h:].double() * _exp2(_per_row(s["x"])).reshape(-1, 1, 1)
    mant, exp = _round(value, "row", most=7)
    mant = mant.to(torch.int32) & 15
    byte = (mant[..., 0::2] | (mant[..., 1::2] << 4)).to(torch.uint8)
    keep = s["slots"] >= 0
    at = s["slots"][keep].long()
    for name, part in (("k", slice(0, kv)), ("v", slice(kv, 2 * kv))):
        s[name].view(-1, kv, d // 2)[at] = byte[keep][:, part]
        s[name + "e"].view(-1, kv)[at] = exp[..., 0][keep][:, part]
    return dict(k=s["k"], v=s["v"], ke=s["ke"], ve=s["ve"])


def _unpack(x):
    """4-bit mantissas, two to a byte, the even one below, as float32."""
    c = x.to(torch.int32)
    c = torch.stack([c & 15, c >> 4], dim=-1).reshape(*x.shape[:-1], -1)
    return ((c ^ 8) - 8).float()


def _cache(case, s):
    n, h, kv, d, page = case["n"], case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    g = h // kv
    blocks = max(1, -(-int(s["pages"].shape[1]) * page // BLOCK))
    at = torch.arange(blocks * BLOCK, device=DEV)
    live = at[None] < s["lengths"][:, None].long()
    slot = s["pages"][:, (at // page).clamp_max(s["pages"].shape[1] - 1)].long().clamp_min(0) * page + at % page
    live = live.reshape(n, blocks, BLOCK)

    def keys(name):
        c = _unpack(s[name].view(-1, kv, d // 2)[slot]).reshape(n, blocks, BLOCK, kv, d).permute(0, 3, 1, 2, 4)
        e = _clip(s[name + "e"].view(-1, kv)[slot]).reshape(n, blocks, BLOCK, kv).permute(0, 3, 1, 2)
        return c.contiguous(), e

    (k, ke), (v, ve) = keys("k"), keys("v")
    q = s["x"][0][:, :h * d].float().reshape(n, kv, 1, g, d).expand(n, kv, blocks, g, d).contiguous()
    c = torch.tensor(s["scale"] * math.log2(math.e), device=DEV, dtype=torch.float64).float()
    r = (c.double() * _exp2(_clip(_per_row(s["x"])))).float().reshape(n, 1, 1, 1, 1)
    see = live[:, None, :, None, :]
    t = (q @ k.transpose(3, 4).contiguous()) * _exp2(ke)[:, :, :, None, :].float()
    t = torch.where(see, t, -math.inf)
    m = t.amax(dim=4, keepdim=True)
    some = live.any(dim=2)[:, None, :, None, None]
    w = torch.where(see, _weight((t - torch.where(some, m, 0.0)).clamp_min(-3e38), r), 0.0).double()
    count = torch.round(w).sum(dim=4, keepdim=True)
    eb = torch.where(live[:, None], ve, E_LO).amax(dim=3)
    num = torch.round(w * _exp2(ve - eb[..., None])[:, :, :, None, :]) @ v.double()
    top, e = m.amax(dim=2, keepdim=True), torch.where(some[..., 0, 0], eb, E_LO).amax(dim=2)
    a = torch.where(some, _weight((m - torch.where(top == -math.inf, 0.0, top)).clamp_min(-3e38), r), 0.0).double()
    total = (torch.round(a) * count).sum(dim=2)
    y = (torch.round(a * _exp2(eb - e[..., None])[:, :, :, None, None]) * num).sum(dim=2)
    y = y * (1.0 / total.clamp_min(1.0)) * _exp2(e)[:, :, None, None]
    mant, exp = _round(y.reshape(n, h * d), "row")
    return dict(mant=mant, exp=exp.reshape(-1))


_PLAIN = dict(rope=_rope, attn_fwd=_attn_fwd, attn_bwd=_attn_bwd, store=_store, cache=_cache)


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def _own(case, s):
    from integer_only_dnn_amd import ie
    h, op = s["h"], case["op"]
    if op == "rope":
        ie.ie_rope(h["rope"], h["x"], s["pos"], h["y"], case["heads"] + case["kv_heads"], h["ws"], inverse=case["inverse"])
        return dict(mant=h["y"].mant, exp=h["y"].exp)
    if op == "attn_fwd":
        ie.ie_attention_fwd(h["plan"], h["x"], h["o"], h["ws"], stats=h["stats"])
        out = dict(mant=h["o"].mant, exp=h["o"].exp)
        if case["stats"]:
            out["stats"] = h["stats"]
        return out
    if op == "attn_bwd":
        ie.ie_attention_bwd(h["plan"], h["x"], h["o"], h["dy"], s["stats"], h["dx"], h["ws"])
        return dict(mant=h["dx"].mant, exp=h["dx"].exp)
    if op == "store":
        ie.ie_cache_store(h["cache"], h["x"], case["heads"], s["slots"], h["ws"])
        return dict(k=s["k"], v=s["v"], ke=s["ke"], ve=s["ve"])
    ie.ie_attention_cache(h["plan"], h["x"], h["cache"], s["pages"], s["lengths"], h["o"], h["ws"])
    return dict(mant=h["o"].mant, exp=h["o"].exp)


def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return _PLAIN[case["op"]](case, state)


def work(case):
    op, h, kv, d = case["op"], case["heads"], case["kv_heads"], case["head_dim"]
    width = (h + 2 * kv) * d
    if op == "rope":
        rows = case["rows"]
        return dict(bytes=2 * rows * (width + 1) + 4 * rows + 2 * case["rot"] * min(rows, case["far"]),
                    flops=3 * rows * (h + kv) * case["rot"])
    if op == "store":
        rows = case["rows"]
        return dict(bytes=rows * (2 * kv * d + 5) + rows * kv * (d + 2), flops=4 * rows * kv * d)
    lengths = _lengths(case)
    if op == "cache":
        return dict(bytes=sum(lengths) * kv * (d + 2) + case["n"] * (2 * h * d + 6) + 4 * sum(-(-t // case["page"]) for t in lengths),
                    flops=4 * sum(lengths) * h * d)
    pairs = sum(t * (t + 1) // 2 if case["causal"] else t * t for t in lengths) * h
    rows = sum(lengths)
    if op == "attn_fwd":
        return dict(bytes=rows * (width + h * d + 2 + (8 * h if case["stats"] else 0)), flops=4 * d * pairs)
    return dict(bytes=rows * (2 * width + 2 * h * d + 8 * h + 4), flops=10 * d * pairs)


# --------------------------------------------------------------------------
# The same from the definition, one sequence and one head after the other, in 64 bits
# --------------------------------------------------------------------------

def _two(x):
    """2^x, exact."""
    return ((x.to(torch.int64) + 1023) * (1 << 52)).view(torch.float64)


def _single(x):
    return x.to(torch.float32).to(torch.float64)


def _pow_fixed(x):
    """The weights of exponents x <= 0 (64 bits, exact products): see the contract at the top."""
    steps = torch.round(torch.clamp(x, min=-64.0) * 131072.0).to(torch.int64).clamp_min(-32 * 131072)
    whole, part = steps >> 17, (steps & 131071).double() / 131072.0
    q = torch.full_like(part, POLY[0])
    for c in POLY[1:]:
        q = _single(q * part + c)
    return q * _two(whole)


def _group(y, most):
    """Mantissas and exponent of one group."""
    top = float(y.abs().max()) if y.numel() else 0.0
    e = -128
    if top > 0.0:
        e = max(math.frexp(top)[1] - most.bit_length() - 1, -128)
        while float(np.rint(math.ldexp(top, -e))) > most:
            e += 1
    return torch.round(y * 2.0 ** -e).to(torch.int8), e


def _grouped(y, group, most=127):
    """The same for every row [rows x cols] or for the whole of it."""
    if group != "row":
        c, e = _group(y, most)
        return c, torch.tensor([e], dtype=torch.int8, device=y.device)
    top = y.abs().amax(dim=1)
    e = torch.full_like(top, -128.0)
    for cand in (1, 0):
        at = torch.frexp(top)[1].double() - most.bit_length() + cand
        fits = torch.round(top * _two(-at)) <= most
        e = torch.where(fits & (top > 0), at, e)
    e = e.clamp_min(-128)
    return torch.round(y * _two(-e)[:, None]).to(torch.int8), e.to(torch.int8)


def _row_exps(t):
    return t[1].double().reshape(-1).expand(t[0].shape[0])


def _spans(case):
    at = 0
    for t in _lengths(case):
        yield at, at + t
        at += t


def _exact_rope(case, s):
    d, rot = case["head_dim"], case["rot"]
    x = s["x"][0].double()
    rows = x.shape[0]
    angle = s["pos"].double()[:, None] * torch.tensor(_frequencies(case)[0], dtype=torch.float64, device=x.device)[None]
    cos, sin = torch.round(torch.cos(angle) * 16384), torch.round(torch.sin(angle) * 16384)
    sin = -sin if case["inverse"] else sin
    y = x * 16384
    for head in range(case["heads"] + case["kv_heads"]):
        k = torch.arange(rot // 2, device=x.device)
        i, j = (2 * k, 2 * k + 1) if case["interleaved"] else (k, k + rot // 2)
        i, j = i + head * d, j + head * d
        y[:, i], y[:, j] = x[:, i] * cos - x[:, j] * sin, x[:, i] * sin + x[:, j] * cos
    mant, exp = _grouped(y * _two(_row_exps(s["x"]) - 14)[:, None], case["group"])
    return dict(mant=mant.reshape(rows, -1), exp=exp)


def _exact_attn(case, s):
    h, kv, d = case["heads"], case["kv_heads"], case["head_dim"]
    x, rows = s["x"][0].double(), s["x"][0].shape[0]
    e = _row_exps(s["x"]).clamp(E_LO, E_HI)
    c = float(np.float32(s["scale"] * math.log2(math.e)))
    back = case["op"] == "attn_bwd"
    y = torch.zeros(rows, (h + 2 * kv if back else h) * d, dtype=torch.float64, device=x.device)
    stats = torch.zeros(rows, h, 2, dtype=torch.int32, device=x.device)
    for a, b in _spans(case):
        f, i = _two(e[a:b]), torch.arange(b - a, device=x.device)
        mask = (i[:, None] >= i[None]) if case["causal"] else torch.ones(b - a, b - a, dtype=torch.bool, device=x.device)
        for hk in range(kv):
            k, v = (x[a:b, (h + z * kv + hk) * d:(h + z * kv + hk + 1) * d] for z in (0, 1))
            mine = []
            for head in range(hk * (h // kv), (hk + 1) * (h // kv)):
                q = x[a:b, head * d:(head + 1) * d]
                t = (q @ k.t().contiguous()) * f[None]
                if back:
                    m = s["stats"][a:b, head, 0].contiguous().view(torch.float32).double()
                else:
                    m = torch.where(mask, t, -math.inf).amax(dim=1)
                w = torch.where(mask, _pow_fixed(torch.clamp(_single(t - m[:, None]), max=0.0) * (c * f)[:, None]), 0.0)
                total = torch.round(w).sum(dim=1)
                if not back:
                    top = torch.where(mask, e[None, a:b], -1e3).amax(dim=1)
                    p = torch.round(w * _two(e[None, a:b] - top[:, None]))
                    y[a:b, head * d:(head + 1) * d] = (p @ v) * (1.0 / total)[:, None] * _two(top)[:, None]
                    stats[a:b, head, 0], stats[a:b, head, 1] = m.float().view(torch.int32), total.to(torch.int32)
                else:
                    mine.append((head, q, w, total))
            if back:
                _exact_heads(case, s, a, b, mine, k, v, e[a:b], mask, y, hk)
    mant, exp = _grouped(y, "row")
    out = dict(mant=mant, exp=exp)
    if case.get("stats"):
        out["stats"] = stats
    return out


def _exact_heads(case, s, a, b, mine, k, v, e, mask, y, hk):
    """Gradients of the heads of one sequence that share keys and values."""
    h, kv, d = case["heads"], case["kv_heads"], case["head_dim"]
    size = lambda z: (torch.frexp((z * z).sum(dim=1))[1].double() + 1).div(2).floor()  # noqa: E731  2^size bounds a row's norm
    ed, eo = _row_exps(s["dy"])[a:b], _row_exps(s["o"])[a:b].clamp(E_LO, E_HI)
    most = ed.max()
    norm = size(v) + e
    parts = []
    for head, q, w, total in mine:
        dy, o = (s[z][0][a:b, head * d:(head + 1) * d].double() for z in ("dy", "o"))
        dot = (dy * o).sum(dim=1)
        u = _single((dy @ v.t().contiguous()) * _two(e)[None] - (dot * _two(eo))[:, None])
        beta, delta = size(dy), torch.frexp(dot.abs())[1].double() + eo
        rise = torch.maximum(beta + (norm + e).max(), delta + e.max()) + 1
        su = _single(w * u)
        n = torch.round(su * _two(e)[None] * _two(-rise)[:, None]) @ k
        y[a:b, head * d:(head + 1) * d] = n * (s["scale"] / total)[:, None] * _two(rise + ed)[:, None]
        share = _single(1.0 / total) * _two((ed - most).clamp_min(-60))
        alpha = torch.frexp(share)[1].double()
        parts.append((q, w, su, dy, share, alpha, alpha + e + torch.maximum(beta + norm.max(), delta) + 1))
    wide = lambda z: torch.where(mask, z[:, None], -1e3).amax(dim=0)  # noqa: E731  over the queries that see a key
    kappa = torch.stack([wide(p[5]) for p in parts]).amax(dim=0)
    lam = torch.stack([wide(p[6]) for p in parts]).amax(dim=0)
    whole = lam.max()
    lam = (lam - whole).clamp_min(-96)
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    for q, w, su, dy, share, alpha, _ in parts:
        dv += torch.round(_single(w * share[:, None]) * _two(-kappa)[None]).t().contiguous() @ dy
        dk += torch.round(_single(su * _single(share * _two(e - whole))[:, None]) * _two(6 - lam)[None]).t().contiguous() @ q
    at = (h + hk) * d
    y[a:b, at:at + d] = dk * s["scale"] * _two(lam - 6 + whole + most)[:, None]
    at += kv * d
    y[a:b, at:at + d] = dv * _two(kappa + most)[:, None]


def _nibbles(row):
    c = row.to(torch.int64)
    c = torch.stack([c % 16, c // 16], dim=-1).reshape(*row.shape[:-1], -1)
    return torch.where(c > 7, c - 16, c).double()


def _exact_store(case, s):
    h, kv, d = case["heads"], case["kv_heads"], case["head_dim"]
    at = torch.nonzero(s["slots"] >= 0).reshape(-1)
    slot = s["slots"][at].long()
    out = {z: s[z].clone() for z in ("k", "v", "ke", "ve")}
    for name, first in (("k", h), ("v", h + kv)):
        for hk in range(kv):
            x = s["x"][0][at, (first + hk) * d:(first + hk + 1) * d].double() * _two(_row_exps(s["x"])[at])[:, None]
            c, e = _grouped(x, "row", 7)
            c = torch.remainder(c.to(torch.int64), 16)
            out[name].view(-1, kv, d // 2)[slot, hk] = (c[:, 0::2] + 16 * c[:, 1::2]).to(torch.uint8)
            out[name + "e"].view(-1, kv)[slot, hk] = e
    return out


def _exact_cache(case, s):
    h, kv, d, page = case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    x = s["x"][0].double()
    y = torch.zeros(case["n"], h * d, dtype=torch.float64, device=x.device)
    c = float(np.float32(s["scale"] * math.log2(math.e)))
    e = _row_exps(s["x"]).clamp(E_LO, E_HI)
    for i, length in enumerate(_lengths(case)):
        if length == 0:
            continue
        j = torch.arange(length, device=x.device)
        slot = s["pages"][i].long()[j // page] * page + j % page
        k, v = (_nibbles(s[z].view(-1, kv, d // 2)[slot]) for z in ("k", "v"))
        ke, ve = (s[z].view(-1, kv)[slot].double().clamp(E_LO, E_HI) for z in ("ke", "ve"))
        q = x[i, :h * d].reshape(kv, h // kv, d)
        t = torch.stack([(q[z] @ k[:, z].t().contiguous()) * _two(ke[:, z])[None] for z in range(kv)])  # [kv, group, keys]
        blocks = [slice(b, min(b + BLOCK, length)) for b in range(0, length, BLOCK)]
        tops, ebs = [t[..., b].amax(dim=2) for b in blocks], [ve[b].amax(dim=0) for b in blocks]
        top, eb = torch.stack(tops).amax(dim=0), torch.stack(ebs).amax(dim=0)
        r = c * _two(e[i])
        total, num = 0.0, 0.0
        for b, m, em in zip(blocks, tops, ebs):
            w = _pow_fixed(_single(t[..., b] - m[..., None]) * r)
            a = _pow_fixed(_single(m - top) * r)
            total = total + torch.round(a) * torch.round(w).sum(dim=2)
            p = torch.round(w * _two(ve[b] - em[None]).t()[:, None])
            num = num + torch.round(a * _two(em - eb)[:, None])[..., None] * (p @ v[b].transpose(0, 1).contiguous())
        y[i] = (num * (1.0 / total)[..., None] * _two(eb)[:, None, None]).reshape(-1)
    mant, exp = _grouped(y, "row")
    return dict(mant=mant, exp=exp)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    if case["op"] == "store":
        return _exact_store(case, s)
    if case["op"] == "cache":
        return _exact_cache(case, s)
    return _exact_attn(case, s)
