"""What is measured of the transformer block's operators on (C, e) tensors.

Layer norm (forward and backward), the forward product with bias, ReLU and
residual in its epilogue, the bias gradient, and dropout from a counter-based
generator (with and without the residual sum).  Every tensor is a pair of int8
mantissas C and int8 exponents e, value C * 2^e; an output comes back as both,
whole numbers that have to be equal bit for bit.

The arithmetic is fixed by the library's contract: int8 products and sums are
exact integers, what cannot be an integer (a row's 1 / sigma, a sum of terms
whose exponents lie far apart) is held to 53 bits, each operation rounded half
to even, and a result is rounded into its groups at the end, at the smallest
exponent that holds the group's largest value.  The plain form below computes
it with elementary torch operations in 64 bits, which are exact or rounded in
just that way.
"""

import math

import numpy as np
import torch

own = False

# Fraction bits of the normalised rows in the two reductions of layer norm's
# backward pass.
FRAC = 20
EPS = (85, -23)  # 1.013e-5, as a (C, e) scalar
DEV = "cuda"


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # the smallest layer of the library's own configurations: latency
        dict(name="norm_fwd_64x256", op="norm_fwd", rows=64, cols=256, group="tensor", affine="tensor"),
        # every token of a ViT-B batch of 128 images, one exponent per token
        dict(name="norm_fwd_25216x768", op="norm_fwd", rows=25216, cols=768, group="row", affine="channel"),
        # a training step's backward through a ViT-Ti batch of 256 images
        dict(name="norm_bwd_50432x192", op="norm_bwd", rows=50432, cols=192, group="row", affine="channel"),
        # few long rows of an odd length, a ragged batch of a wide model
        dict(name="norm_bwd_1031x4099", op="norm_bwd", rows=1031, cols=4099, group="tensor", affine="tensor"),
        # bias + ReLU of the smallest layer: latency
        dict(name="linear_64x128x256", op="linear", rows=64, cols=128, inner=256, group="tensor", w="tensor",
             bias="tensor", relu=True, residual="none"),
        # ViT-Ti's first MLP product: short contraction, rows wider than a tile
        dict(name="linear_50432x768x192", op="linear", rows=50432, cols=768, inner=192, group="row", w="row",
             bias="channel", relu=True, residual="none"),
        # ViT-B's attention projection back onto the residual stream
        dict(name="linear_25216x768x768", op="linear", rows=25216, cols=768, inner=768, group="row", w="row",
             bias="channel", relu=False, residual="row"),
        # a few tokens being answered through a wide layer: the weight is what is read
        dict(name="linear_5x4096x4096", op="linear", rows=5, cols=4096, inner=4096, group="row", w="row",
             bias="channel", relu=False, residual="row"),
        # the bias gradient of ViT-B's MLP input over a batch
        dict(name="bias_grad_25216x2304", op="bias_grad", rows=25216, cols=2304, group="row", affine="channel"),
        # dropout of a sublayer's output, added onto the residual stream
        dict(name="dropout_25216x768", op="dropout", rows=25216, cols=768, group="row", out="row", drop=6554,
             residual="row"),
        # its gradient: the same draws, whole-tensor exponent
        dict(name="dropout_16384x1024", op="dropout", rows=16384, cols=1024, group="tensor", out="tensor", drop=6554,
             residual="none"),
        # attention rows of odd length, half of them dropped
        dict(name="dropout_591x197", op="dropout", rows=591, cols=197, group="row", out="row", drop=32768,
             residual="none"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "linear", "linear", "bias_grad", "dropout"])
    group = rng.choice(["row", "row", "tensor"])
    affine = rng.choice(["channel", "tensor"])
    if op == "linear":
        while True:
            rows, cols, inner = _log(rng, 1, 50432), _log(rng, 1, 8192), _log(rng, 1, 8192)
            if rows * cols <= 24_000_000 and rows * cols * inner <= 14_000_000_000 and rows * inner <= 30_000_000:
                break
        return dict(op=op, rows=rows, cols=cols, inner=inner, group=group, w=rng.choice(["row", "tensor"]),
                    bias=rng.choice(["channel", "tensor", "none"]), relu=rng.random() < 0.5,
                    residual=rng.choice(["row", "tensor", "none"]))
    while True:
        rows, cols = _log(rng, 1, 50432), _log(rng, 1, 16384)
        if 64 <= rows * cols <= 16_000_000:
            break
    if op in ("norm_fwd", "norm_bwd"):
        return dict(op=op, rows=rows, cols=cols, group=group, affine=rng.choice(["channel", "tensor", "none"]))
    if op == "bias_grad":
        return dict(op=op, rows=rows, cols=cols, group=group, affine=affine)
    return dict(op=op, rows=rows, cols=cols, group=group, out=rng.choice(["row", "tensor"]),
                drop=rng.choice([0, 3277, 6554, 13107, 32768, 49152]), residual=rng.choice(["row", "tensor", "none"]))


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _quantise(x, group):
    """(C, e) of real values: each group's largest magnitude becomes 127."""
    mx = x.abs().amax(dim=1, keepdim=True) if group != "tensor" else x.abs().max().reshape(1, 1)
    mx = mx.clamp_min(1e-30)
    c = torch.round(x * (127.0 / mx)).to(torch.int8)
    e = (torch.ceil(torch.log2(mx)) - 7).to(torch.int8).reshape(-1)
    return c.contiguous(), e.contiguous()


def _tokens(g, rows, cols, group, scale=1.0, pad=False):
    """Activations or gradients whose rows differ in size, as a network's do; `pad`: some rows are padding, all zero."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x = x * (scale * torch.exp2(torch.randn(rows, 1, generator=g, device=DEV)))
    if pad:
        x[torch.arange(rows, device=DEV) % 64 == 63] = 0
    return _quantise(x, group)


def _vector(g, n, kind, mean, spread):
    """A parameter of n channels, [n x 1]: one exponent, or one per channel."""
    x = mean + spread * torch.randn(n, 1, generator=g, device=DEV)
    return _quantise(x, "tensor" if kind == "tensor" else "row")


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, rows, cols, group = case["op"], case["rows"], case["cols"], case["group"]
    s = dict(case=case)
    if op in ("norm_fwd", "norm_bwd"):
        s["x"] = _tokens(g, rows, cols, group, pad=True)
        if case["affine"] != "none":
            s["gamma"] = _vector(g, cols, case["affine"], 1.0, 0.2)
            s["beta"] = _vector(g, cols, case["affine"], 0.0, 0.3)
        if op == "norm_bwd":
            s["dy"] = _tokens(g, rows, cols, group, scale=2.0 ** -10)
    elif op == "linear":
        s["x"] = _tokens(g, rows, case["inner"], group)
        w = torch.randn(cols, case["inner"], generator=g, device=DEV) * case["inner"] ** -0.5
        s["w"] = _quantise(w, case["w"])
        if case["bias"] != "none":
            s["bias"] = _vector(g, cols, case["bias"], 0.0, 0.3)
        if case["residual"] != "none":
            s["r"] = _tokens(g, rows, cols, case["residual"], scale=2.0)
    elif op == "bias_grad":
        s["dy"] = _tokens(g, rows, cols, group, scale=2.0 ** -10)
    else:
        s["x"] = _tokens(g, rows, cols, group)
        s["seed"], s["step"] = seed * 0x9E3779B97F4A7C15 % (1 << 64), seed % 1000
        if case["residual"] != "none":
            s["r"] = _tokens(g, rows, cols, case["residual"], scale=2.0)
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program that uses the library keeps: its tensors as (C, e) matrices, the outputs, a workspace."""
    from integer_only_dnn_amd import ie
    case = s["case"]
    op, rows, cols = case["op"], case["rows"], case["cols"]

    def mat(key, group):
        if key not in s:
            return None
        return ie.Mat(s[key][0], s[key][1], ie.TENSOR if group == "tensor" else ie.ROW)

    def out(r, c, group):
        return ie.Mat.empty(r, c, ie.TENSOR if group == "tensor" else ie.ROW, DEV)

    h = dict(ws=ie.Workspace(DEV), x=mat("x", case["group"]), dy=mat("dy", case["group"]))
    vec = case.get("affine", case.get("bias"))
    h["gamma"], h["beta"], h["bias"] = mat("gamma", vec), mat("beta", vec), mat("bias", vec)
    h["w"], h["r"] = mat("w", case.get("w")), mat("r", case.get("residual"))
    if op == "bias_grad":
        h["db"] = out(cols, 1, vec)
    elif op == "norm_bwd":
        h["dx"] = out(rows, cols, case["group"])
        if vec != "none":
            h["dgamma"], h["dbeta"] = out(cols, 1, vec), out(cols, 1, vec)
    else:
        h["y"] = out(rows, cols, case.get("out", case["group"]))
    s["h"] = h


# --------------------------------------------------------------------------
# The plain form: elementary torch operations in 64 bits
# --------------------------------------------------------------------------

def _exp2(e):
    """2^e in float64, exactly (e an integer tensor within the normal range)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _value(t):
    """(C, e) as float64, exact."""
    c, e = t
    return c.double() * _exp2(e.reshape(-1, 1) if e.numel() > 1 else e.reshape(1, 1))


def _round(y, group):
    """Values into int8 groups: the smallest exponent that holds the group's largest magnitude, ties to even."""
    mx = y.abs().amax(dim=1, keepdim=True) if group != "tensor" else y.abs().max().reshape(1, 1)
    _, x = torch.frexp(mx)
    e = x.to(torch.int64) - 7
    e = torch.where(torch.round(mx * _exp2(-e)) > 127, e + 1, e)
    e = torch.where(mx == 0, torch.full_like(e, -128), e).clamp_min(-128)
    c = torch.round(y * _exp2(-e)).to(torch.int8)
    return dict(mant=c, exp=e.reshape(-1).to(torch.int8))


def _align(t):
    """Mantissas re-expressed at the largest exponent (exact integers in float64), and that exponent."""
    c, e = t
    top = e.max()
    s = (e.to(torch.int64) - top.to(torch.int64)).clamp_min(-64)
    return torch.round(c.double() * _exp2(s).reshape(-1, 1)), top.to(torch.int64)


def _rows(case, x):
    """A row's exact sums: N C - sum C of every element, and 1 / sqrt of N^2 times (its variance + eps)."""
    c, e = x[0].double(), x[1].reshape(-1, 1).to(torch.int64)
    n = float(case["cols"])
    total, squares = c.sum(dim=1, keepdim=True), (c * c).sum(dim=1, keepdim=True)
    spread = n * squares - total * total
    t = spread + n * n * EPS[0] * _exp2(EPS[1] - 2 * e)
    return n * c - total, 1.0 / torch.sqrt(t)


def _norm_fwd(case, s):
    d, r = _rows(case, s["x"])
    y = d * r
    if "gamma" in s:
        y = y * _value(s["gamma"]).reshape(1, -1)
        y = y + _value(s["beta"]).reshape(1, -1)
    return _round(y, case["group"])


def _norm_bwd(case, s):
    n, x, dy = float(case["cols"]), s["x"], s["dy"]
    d, r = _rows(case, x)
    f = torch.round(d * r * 2.0 ** FRAC)
    g, top = dy[0].double(), 0
    if "gamma" in s:
        gamma, top = _align(s["gamma"])
        g = g * gamma.reshape(1, -1)
    g1, g2 = g.sum(dim=1, keepdim=True), (g * f).sum(dim=1, keepdim=True)
    z = (n * g - g1) - f * (g2 * 2.0 ** (-2 * FRAC))
    scale = _exp2(dy[1].to(torch.int64).reshape(-1, 1) + top - x[1].to(torch.int64).reshape(-1, 1))
    out = dict(dx=_round(z * r * scale, case["group"]))
    if "gamma" in s:
        a, at = _align(dy)
        out["dgamma"] = _round((a * f).sum(dim=0).reshape(-1, 1) * _exp2(at - FRAC), case["affine"])
        out["dbeta"] = _round(a.sum(dim=0).reshape(-1, 1) * _exp2(at), case["affine"])
    return out


def _linear(case, s):
    acc = s["x"][0].double() @ s["w"][0].double().t()
    y = acc * _exp2(s["x"][1]).reshape(-1, 1) * _exp2(s["w"][1]).reshape(1, -1)
    if "bias" in s:
        y = y + _value(s["bias"]).reshape(1, -1)
    if "r" in s:
        y = y + _value(s["r"])
    out = _round(y, case["group"])
    if case["relu"]:
        out["mant"] = out["mant"].clamp_min(0)
    return out


def _draws(rows, cols, seed, step):
    """Sixteen random bits per element: Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011) under key `seed`, one block
    of 128 bits for eight neighbours of a row, counter (column / 8, row, step)."""
    m = 0xFFFFFFFF
    blocks = (cols + 7) // 8
    c0 = torch.arange(blocks, device=DEV).reshape(1, -1).expand(rows, blocks)
    c1 = torch.arange(rows, device=DEV).reshape(-1, 1).expand(rows, blocks)
    c2, c3 = torch.full_like(c0, step & m), torch.full_like(c0, step >> 32)
    k0, k1 = seed & m, seed >> 32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (p1 >> 32) & m ^ c1 ^ k0, p1 & m, (p0 >> 32) & m ^ c3 ^ k1, p0 & m
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    words = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16], 2)
    return words.reshape(rows, blocks * 8)[:, :cols]


def _dropout(case, s):
    keep = _draws(case["rows"], case["cols"], s["seed"], s["step"]) >= case["drop"]
    scale = float(np.float32(65536.0 / (65536 - case["drop"])))
    y = torch.where(keep, _value(s["x"]) * scale, 0.0)
    if "r" in s:
        y = y + _value(s["r"])
    return _round(y, case["out"])


def _bias_grad(case, s):
    a, at = _align(s["dy"])
    return _round(a.sum(dim=0).reshape(-1, 1) * _exp2(at), case["affine"])


_PLAIN = dict(norm_fwd=_norm_fwd, norm_bwd=_norm_bwd, linear=_linear, dropout=_dropout, bias_grad=_bias_grad)


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def _pair(m):
    return dict(mant=m.mant, exp=m.exp)


def _own(case, s):
    from integer_only_dnn_amd import ie
    h, op = s["h"], case["op"]
    if op == "norm_fwd":
        ie.ie_layer_norm_fwd(h["x"], h["gamma"], h["beta"], EPS, h["y"], h["ws"])
    elif op == "norm_bwd":
        ie.ie_layer_norm_bwd(h["dy"], h["x"], h["gamma"], EPS, h["dx"], h.get("dgamma"), h.get("dbeta"), h["ws"])
        out = dict(dx=_pair(h["dx"]))
        if "dgamma" in h:
            out["dgamma"], out["dbeta"] = _pair(h["dgamma"]), _pair(h["dbeta"])
        return out
    elif op == "linear":
        ie.ie_linear_fwd_fused(h["x"], h["w"], h["bias"], h["r"], h["y"],
                               ie.ACT_RELU if case["relu"] else ie.ACT_NONE, h["ws"])
    elif op == "bias_grad":
        ie.ie_linear_bwd_db(h["dy"], h["db"], h["ws"])
        return _pair(h["db"])
    else:
        ie.ie_dropout(h["x"], h["r"], h["y"], case["drop"], s["seed"], s["step"], h["ws"])
    return _pair(h["y"])


def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return _PLAIN[case["op"]](case, state)


def work(case):
    op, m, n = case["op"], case["rows"], case["cols"]
    tall = lambda kind: m if kind == "row" else 1  # noqa: E731  exponents of an activation
    vec = {"channel": 2 * n, "tensor": n, "none": 0}
    if op == "norm_fwd":
        return dict(bytes=2 * (m * n + tall(case["group"])) + 2 * vec[case["affine"]], flops=8 * m * n)
    if op == "norm_bwd":
        return dict(bytes=3 * (m * n + tall(case["group"])) + 3 * vec[case["affine"]], flops=18 * m * n)
    if op == "linear":
        k = case["inner"]
        res = m * n if case["residual"] != "none" else 0
        return dict(bytes=m * k + n * k + m * n + res + vec[case["bias"]] + 2 * tall(case["group"]) + n,
                    flops=2 * m * n * k)
    if op == "bias_grad":
        return dict(bytes=m * n + tall(case["group"]) + vec[case["affine"]], flops=m * n)
    res = m * n if case["residual"] != "none" else 0
    return dict(bytes=2 * m * n + res + 2 * tall(case["group"]), flops=4 * m * n)


# --------------------------------------------------------------------------
# The same from the definition, in numpy, 64-bit integers where it can be
# --------------------------------------------------------------------------

def _host(t):
    return t[0].cpu().numpy().astype(np.int64), t[1].cpu().numpy().astype(np.int64).reshape(-1, 1)


def _np_round(y, group):
    mx = np.max(np.abs(y), axis=1, keepdims=True) if group != "tensor" else np.max(np.abs(y)).reshape(1, 1)
    e = np.frexp(mx)[1].astype(np.int64) - 7
    e = e + (np.rint(np.ldexp(mx, -e)) > 127)
    e = np.maximum(np.where(mx == 0, -128, e), -128)
    return dict(mant=np.rint(np.ldexp(y, -e)).astype(np.int8), exp=e.reshape(-1).astype(np.int8))


def _np_align(c, e):
    return np.rint(np.ldexp(c.astype(np.float64), np.maximum(e - e.max(), -64))).astype(np.int64), int(e.max())


def _np_rows(case, x):
    c, e = _host(x)
    n = case["cols"]
    total = c.sum(axis=1, keepdims=True)
    spread = n * (c * c).sum(axis=1, keepdims=True) - total * total
    t = spread.astype(np.float64) + np.ldexp(np.float64(n * n * EPS[0]), EPS[1] - 2 * e)
    return n * c - total, 1.0 / np.sqrt(t)


def _np_philox(rows, cols, seed, step):
    m, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    blocks = (cols + 7) // 8
    c = [np.tile(np.arange(blocks, dtype=np.uint64), rows), np.repeat(np.arange(rows, dtype=np.uint64), blocks),
         np.full(rows * blocks, step & 0xFFFFFFFF, np.uint64), np.full(rows * blocks, step >> 32, np.uint64)]
    for i in range(10):
        k = [((seed & 0xFFFFFFFF) + i * 0x9E3779B9) % (1 << 32), ((seed >> 32) + i * 0xBB67AE85) % (1 << 32)]
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> sh) ^ c[1] ^ np.uint64(k[0]), b & m, (a >> sh) ^ c[3] ^ np.uint64(k[1]), a & m]
    u = np.stack(c, axis=1).astype(np.uint32).view(np.uint16)  # low half first
    return u.reshape(rows, blocks * 8)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op, group = case["op"], case["group"]

    def val(key):
        c, e = _host(s[key])
        return np.ldexp(c.astype(np.float64), e)

    if op == "linear":
        (xc, xe), (wc, we) = _host(s["x"]), _host(s["w"])
        y = np.ldexp(np.matmul(xc.astype(np.float64), wc.T.astype(np.float64)), xe + we.reshape(1, -1))
        if "bias" in s:
            y = y + val("bias").reshape(1, -1)
        if "r" in s:
            y = y + val("r")
        out = _np_round(y, group)
        if case["relu"]:
            out["mant"] = np.maximum(out["mant"], 0)
        return out
    if op == "bias_grad":
        a, at = _np_align(*_host(s["dy"]))
        return _np_round(np.ldexp(a.sum(axis=0).astype(np.float64), at).reshape(-1, 1), case["affine"])
    if op == "dropout":
        keep = _np_philox(case["rows"], case["cols"], s["seed"], s["step"]) >= case["drop"]
        y = val("x") * np.float64(np.float32(65536.0 / (65536 - case["drop"]))) * keep
        return _np_round(y + val("r") if "r" in s else y, case["out"])
    d, r = _np_rows(case, s["x"])
    h = d.astype(np.float64) * r
    if op == "norm_fwd":
        if "gamma" in s:
            h = h * val("gamma").reshape(1, -1) + val("beta").reshape(1, -1)
        return _np_round(h, group)
    n, f = case["cols"], np.rint(np.ldexp(h, FRAC)).astype(np.int64)
    (dc, de), xe = _host(s["dy"]), _host(s["x"])[1]
    g, top = dc, 0
    if "gamma" in s:
        gam, top = _np_align(*_host(s["gamma"]))
        g = dc * gam.reshape(1, -1)
    g1, g2 = g.sum(axis=1, keepdims=True), (g * f).sum(axis=1, keepdims=True)
    z = (n * g - g1).astype(np.float64) - f.astype(np.float64) * np.ldexp(g2.astype(np.float64), -2 * FRAC)
    out = dict(dx=_np_round(np.ldexp(z * r, de + top - xe), group))
    if "gamma" in s:
        a, at = _np_align(dc, de)
        out["dgamma"] = _np_round(np.ldexp((a * f).sum(axis=0).astype(np.float64), at - FRAC).reshape(-1, 1),
                                  case["affine"])
        out["dbeta"] = _np_round(np.ldexp(a.sum(axis=0).astype(np.float64), at).reshape(-1, 1), case["affine"])
    return out
