"""The oracle's attention, rotary positions and 4-bit cache against formulas in
64 bits: softmax in float64, autograd, central differences, complex rotations.
Tolerances are sums of the roundings that the arithmetic names."""

import math

import numpy as np
import pytest
import torch

import oracle as o
from tests.gpu_util import rand_qt

# a weight's relative error: the cubic (checked below), and half of 2^-17 in the
# exponent, (2^(2^-18) - 1) = ln 2 * 2^-18
W_ERR = 1.1e-4 + math.log(2) * 2.0 ** -18 + 4 * 2.0 ** -24


def values(t):
    return np.ldexp(t.mant.astype(np.float64), t.row_exp()[:, None])


def case(seed, rows, heads, kv, d, group=o.ROW, elo=-9, ehi=-5):
    rng = np.random.default_rng(seed)
    X = rand_qt(rng, (rows, (heads + 2 * kv) * d), group, elo, ehi)
    X.mant[:] = np.clip(np.rint(rng.normal(0, 40, X.mant.shape)), -127, 127)
    return rng, X


def test_weight_is_a_power_of_two():
    d = -np.concatenate([[0.0], np.random.default_rng(0).uniform(0, 15, 20000), np.arange(40.0)]).astype(np.float32)
    w = o.softmax_weight(d.astype(np.float64), np.float64(1.0))
    assert w[0] == 32512 and np.all(w <= 32512 * (1 + 1.1e-4))
    near = d > -31
    assert np.abs(w[near] / (32512 * 2.0 ** d[near].astype(np.float64)) - 1).max() <= W_ERR
    assert np.all(np.rint(w[d <= -16]) == 0)
    assert np.all(w[-40:][:32] == 32512 * 2.0 ** -np.arange(32.0))  # whole exponents are exact
    assert np.all(o.softmax_weight(np.float64([-1e30, -3e38]), np.float64(2.0 ** 60)) == 32512 * 2.0 ** -32)


def softmax64(X, heads, kv, d, scale, causal, offsets):
    """(o, p) in float64 from X's values, as torch tensors with a graph."""
    x = torch.from_numpy(values(X)).requires_grad_()
    outs, ps = torch.zeros(x.shape[0], heads * d, dtype=torch.float64), []
    rows = []
    for a, b in zip(offsets[:-1], offsets[1:]):
        if a == b:
            continue
        s = x[a:b].reshape(b - a, heads + 2 * kv, d).transpose(0, 1)
        q, k, v = s[:heads], s[heads:heads + kv].repeat_interleave(heads // kv, 0), s[heads + kv:].repeat_interleave(heads // kv, 0)
        t = q @ k.transpose(1, 2) * scale
        if causal:
            t = t.masked_fill(~torch.ones(b - a, b - a, dtype=torch.bool).tril(), -math.inf)
        p = torch.softmax(t, 2)
        ps.append((a, b, p.detach().numpy(), v.detach().numpy(), k.detach().numpy(), q.detach().numpy()))
        rows.append((a, b, (p @ v).transpose(0, 1).reshape(b - a, heads * d)))
    outs = torch.cat([torch.zeros(0, heads * d, dtype=torch.float64)] + [r for _, _, r in rows])
    return x, outs, ps


CASES = [(1, 1, 1, 8, False, [0, 1]), (13, 2, 1, 8, True, [0, 13]), (40, 4, 2, 16, True, [0, 7, 7, 40]),
         (40, 3, 3, 20, False, [0, 1, 33, 40]), (150, 2, 2, 32, True, [0, 150])]


def forward_bound(X, p, v, L, e, scale):
    """How far a head's o may be from softmax's: weights off by W_ERR relative, twice (numerator and sum), and by half a
    unit each in both sums."""
    vmax = np.abs(v).max(axis=(1, 2))[:, None]
    n = p.shape[2]
    return 2 * W_ERR * np.einsum("hij,hjd->hid", p, np.abs(v)).max(axis=2) + n * (127 * 2.0 ** e.max() + vmax) * 0.5 / L


@pytest.mark.parametrize("group", [o.ROW, o.TENSOR])
@pytest.mark.parametrize("rows,heads,kv,d,causal,offsets", CASES)
def test_forward_against_softmax(rows, heads, kv, d, causal, offsets, group):
    rng, X = case(rows + heads, rows, heads, kv, d, group)
    scale = float(np.float32(d ** -0.5))
    O, tops, sums = o.attention_fwd(X, heads, kv, d, scale, causal, offsets)
    _, want, ps = softmax64(X, heads, kv, d, scale, causal, offsets)
    got = values(O)
    for a, b, p, v, k, q in ps:
        L = sums[a:b].T.astype(np.float64)
        tol = forward_bound(X, p, v, L, X.row_exp()[a:b], scale)  # [heads, rows]
        tol = np.repeat(tol.T[:, :, None], d, axis=2).reshape(b - a, -1) + 0.5 * np.ldexp(1.0, O.row_exp()[a:b])[:, None]
        assert np.all(np.abs(got[a:b] - want.detach().numpy()[a:b]) <= tol)
        # the sums: softmax's denominators
        t = np.einsum("hid,hjd->hij", q, k) * scale
        see = np.tri(b - a, dtype=bool) if causal else np.ones((b - a, b - a), bool)
        den = np.where(see, np.exp(t - np.where(see, t, -np.inf).max(axis=2, keepdims=True)), 0.0).sum(axis=2) * 32512
        # fp32 roundings of the difference, of r and of their product: 2^-24 relative each of at most |t|
        off = 2 ** np.abs(3 * 2.0 ** -24 * np.abs(t).max() * 2 / math.log(2)) - 1
        assert np.all(np.abs(L - den) <= (W_ERR + off) * den + 0.5 * (b - a))


def test_one_token_is_its_value():
    """A softmax over one key: o = v whatever the scores, and dq = dk = 0, dv = dO."""
    rng, X = case(3, 5, 3, 3, 16)
    off = [0, 1, 2, 3, 4, 5]
    O, tops, sums = o.attention_fwd(X, 3, 3, 16, 0.25, True, off)
    assert np.array_equal(values(O), values(o.requant_f64(values(X)[:, 96:], o.ROW))) and np.all(sums == 32512)
    dO = rand_qt(rng, (5, 48), o.ROW, -20, -12)
    G = values(o.attention_bwd(X, O, dO, tops, sums, 3, 3, 16, 0.25, True, off))
    # dv up to the rounding of 1 / L to fp32, the weight's half unit and the row's half unit
    tol = np.abs(values(dO)) * 2.0 ** -14 + 0.5 * np.ldexp(1.0, o.requant_f64(G, o.ROW).row_exp())[:, None]
    assert np.all(np.abs(G[:, 96:] - values(dO)) <= tol)


def test_tokens_do_not_see_later_ones():
    """Whatever a later token holds, and however large its exponent, the results of those before it stay."""
    rng, X = case(8, 30, 2, 1, 16)
    O = o.attention_fwd(X, 2, 1, 16, 0.25, True)[0]
    Y = o.QT(X.mant.copy(), X.exp.copy(), o.ROW)
    Y.mant[20:] = rng.integers(-127, 128, Y.mant[20:].shape)
    Y.exp[20:] += 9
    P = o.attention_fwd(Y, 2, 1, 16, 0.25, True)[0]
    assert np.array_equal(O.mant[:20], P.mant[:20]) and np.array_equal(O.exp[:20], P.exp[:20])
    assert not np.array_equal(O.mant[20:], P.mant[20:])


def test_sequences_are_apart_and_rows_of_none_are_zero():
    rng, X = case(9, 21, 2, 2, 8)
    O = o.attention_fwd(X, 2, 2, 8, 0.5, False, [2, 9, 9, 18])[0]
    for a, b in ((2, 9), (9, 18)):
        one = o.attention_fwd(o.QT(X.mant[a:b], X.exp[a:b], o.ROW), 2, 2, 8, 0.5, False)[0]
        assert np.array_equal(O.mant[a:b], one.mant) and np.array_equal(O.exp[a:b], one.exp)
    for r in (0, 1, 18, 19, 20):
        assert not O.mant[r].any() and O.exp[r] == o.E_MIN


def backward_bound(X, O, dO, o64, a, b, p, v, k, q, L, scale, heads, kv, d, whole):
    """Elementwise bounds of |dQ|, |dK|, |dV| errors before the last rounding."""
    g = heads // kv
    x, dy = X.row_exp()[a:b], values(dO)[a:b].reshape(b - a, heads, d).transpose(1, 0, 2)
    e = np.ldexp(1.0, x)
    dO_ = np.abs(dy)
    off = np.abs(values(O)[a:b] - o64[a:b]).reshape(b - a, heads, d).transpose(1, 0, 2)
    dD = (dO_ * off).sum(axis=2)  # D is taken from the rounded O
    dP = np.einsum("hid,hjd->hij", dy, v)
    u = dP - (p * dP).sum(axis=2, keepdims=True)
    big = np.abs(dP) + np.abs((p * dP).sum(axis=2, keepdims=True))
    # p is off by twice the weight's error and half a unit of the sum's; u by dD and an fp32 rounding
    perr = p * (2 * W_ERR + 0.5 * p.shape[2] / L[:, :, None] + 2.0 ** -22)
    serr = perr * big + (p + perr) * (dD[:, :, None] + 2.0 ** -22 * big)
    return serr, perr, dO_


@pytest.mark.parametrize("group", [o.ROW, o.TENSOR])
@pytest.mark.parametrize("rows,heads,kv,d,causal,offsets", CASES[1:])
def test_backward_against_autograd(rows, heads, kv, d, causal, offsets, group):
    rng, X = case(rows + heads, rows, heads, kv, d, group)
    scale = float(np.float32(d ** -0.5))
    O, tops, sums = o.attention_fwd(X, heads, kv, d, scale, causal, offsets)
    dO = rand_qt(rng, (rows, heads * d), group, -20, -17)
    G = o.attention_bwd(X, O, dO, tops, sums, heads, kv, d, scale, causal, offsets)
    x, y, ps = softmax64(X, heads, kv, d, scale, causal, offsets)
    want, = torch.autograd.grad((y * torch.from_numpy(values(dO)[offsets[0]:offsets[-1]])).sum(), x)
    want, got, g = want.numpy(), values(G), heads // kv
    for a, b, p, v, k, q in ps:
        L = sums[a:b].T.astype(np.float64)
        serr, perr, dabs = backward_bound(X, O, dO, y.detach().numpy(), a, b, p, v, k, q, L, scale, heads, kv, d, offsets)
        e, ed, eo = X.row_exp()[a:b], dO.row_exp()[a:b], O.row_exp()[a:b]
        dq = scale * np.einsum("hij,hjd->hid", serr, np.abs(k))
        dk = scale * np.einsum("hij,hid->hjd", serr, np.abs(q))
        dv = np.einsum("hij,hid->hjd", perr, dabs)
        # half units of the integers A, B, C: their scales are at most 2^2 times the norms' products they stand for
        # (a ceiling of each norm's bits), so with N = the largest norms
        vn = np.linalg.norm(v, axis=2).max(axis=1)[:, None] * 2
        dn = np.linalg.norm(dabs, axis=2) * 2
        dot = np.abs((values(dO)[a:b] * values(O)[a:b]).reshape(b - a, heads, d).sum(axis=2)).T * 2
        unit = 2 * np.maximum(dn * vn, dot) * 127 * np.ldexp(1.0, e.max())  # 2^sigma in values, times |k|
        dq += scale * 0.5 * unit[:, :, None] * (b - a) / L[:, :, None]
        am = (2.0 ** np.maximum(ed - ed.max(), -60) / L).max() * 2 * 2.0 ** ed.max()
        dv += 0.5 * am * np.abs(dO.mant.astype(np.float64)).max() * (b - a)
        lm = (2.0 ** np.maximum(ed - ed.max(), -60) / L * 2 * 2 * np.maximum(dn / 2.0 ** ed * vn, dot / 2.0 ** ed)
              * 2.0 ** e).max() * 2.0 ** ed.max()
        dk += scale * 0.5 * lm / 64 * 127 * (b - a)
        dk, dv = (z.reshape(kv, g, b - a, d).sum(axis=1) for z in (dk, dv))
        tol = np.concatenate([z.transpose(1, 0, 2).reshape(b - a, -1) for z in (dq, dk, dv)], axis=1)
        tol = tol + 0.5 * np.ldexp(1.0, G.row_exp()[a:b])[:, None]
        assert np.all(np.abs(got[a:b] - want[a:b]) <= tol)


def test_backward_against_differences():
    """A directional derivative by central differences of the formula, against the gradient's product with the direction;
    the gradient's error is at most its rounding's and the weights' (bounds as above, as norms)."""
    rng, X = case(5, 24, 2, 1, 16)
    O, tops, sums = o.attention_fwd(X, 2, 1, 16, 0.25, True)
    dO = rand_qt(rng, (24, 32), o.ROW, -8, -6)
    G = values(o.attention_bwd(X, O, dO, tops, sums, 2, 1, 16, 0.25, True))

    def loss(x):
        s = x.reshape(24, 4, 16).transpose(1, 0, 2)
        t = np.einsum("hid,jd->hij", s[:2], s[2]) * 0.25
        t = np.where(np.tri(24, dtype=bool), t, -np.inf)
        p = np.exp(t - t.max(axis=2, keepdims=True))
        y = np.einsum("hij,jd->hid", p / p.sum(axis=2, keepdims=True), s[3])
        return (y.transpose(1, 0, 2).reshape(24, 32) * values(dO)).sum()

    x, h = values(X), 1e-5
    want, _, _ = softmax64(X, 2, 1, 16, 0.25, True, [0, 24])
    for k in range(4):
        v = rng.normal(size=x.shape)
        diff = (loss(x + h * v) - loss(x - h * v)) / (2 * h)
        # half a unit of each of the row's elements, and as much again for D from the rounded O and the weights
        tol = np.sqrt((np.ldexp(1.0, 2 * o.requant_f64(G, o.ROW).row_exp())[:, None] * v * v).sum()) * 4
        assert abs(diff - (G * v).sum()) <= tol


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,d", [(8, 8), (6, 10), (32, 64), (0, 8)])
def test_rope_is_a_rotation(rot, d, interleaved):
    rng = np.random.default_rng(rot + d)
    X = rand_qt(rng, (9, 4 * d), o.ROW, -9, -5)
    pos, f = rng.integers(0, 50000, 9), o.rope_frequencies(rot)
    table = np.zeros((50000, rot // 2, 2), np.int16)
    table[pos] = [o.rope_table(f, int(p) + 1)[-1] for p in pos]
    Y = o.rope(X, pos, table, 3, d, rot, interleaved, False, o.ROW)
    x, y = values(X).reshape(9, 4, d), values(Y).reshape(9, 4, d)
    want = x.copy()
    for k in range(rot // 2):
        i, j = (2 * k, 2 * k + 1) if interleaved else (k, k + rot // 2)
        z = (x[:, :3, i] + 1j * x[:, :3, j]) * np.exp(1j * pos * f[k])[:, None]
        want[:, :3, i], want[:, :3, j] = z.real, z.imag
    unit = np.ldexp(1.0, Y.row_exp())[:, None, None]
    # half a unit of the row, half a unit of 2^-14 of each of two products
    assert np.all(np.abs(y - want) <= 0.5 * unit + 2 * 2.0 ** -15 * np.abs(x).max(axis=(1, 2), keepdims=True))
    Z = o.rope(Y, pos, table, 3, d, rot, interleaved, True, o.ROW)
    back = values(Z).reshape(9, 4, d)
    again = 0.5 * np.ldexp(1.0, Z.row_exp())[:, None, None] + 2 * unit + 8 * 2.0 ** -15 * np.abs(x).max(axis=(1, 2), keepdims=True)
    assert np.all(np.abs(back - x) <= again)


def test_rope_frequencies():
    f = o.rope_frequencies(64)
    assert f[0] == 1.0 and abs(f[16] - 0.01) < 1e-15
    assert np.allclose(o.rope_frequencies(64, factor=4.0), np.array(f) / 4, rtol=1e-15)
    p = o.rope_frequencies(128, factor=8.0, trained=8192.0)
    plain = np.array(o.rope_frequencies(128))
    assert p[0] == plain[0] and p[-1] == plain[-1] / 8  # fast pairs stay, slow ones are stretched
    assert np.all(np.diff(p) < 0) and np.all((np.array(p) <= plain) & (np.array(p) >= plain / 8))
    assert np.array_equal(o.rope_table(f, 1)[0], np.tile([16384, 0], (32, 1)))


def test_four_bit_rows():
    rng = np.random.default_rng(2)
    x = rng.integers(-128, 128, (400, 16))
    x[0], x[1], x[2] = 0, 7, -128
    c, e = o.cache_row(x, np.full(400, -6))
    assert np.abs(c).max() <= 7 and e[0] == o.E_MIN and not c[0].any() and np.all(c[1] == 7) and e[1] == -6
    on = np.arange(400) != 0
    err = np.abs(np.ldexp(c[on].astype(np.float64), e[on, None]) - np.ldexp(x[on].astype(np.float64), -6))
    assert np.all(err <= 0.5 * np.ldexp(1.0, e[on])[:, None])
    assert np.all(np.abs(c[on]).max(axis=1) >= 4)  # the smallest exponent that holds the row
    assert np.array_equal(o.unpack4(o.pack4(c)), c)


@pytest.mark.parametrize("lengths", [[1], [5, 0, 256, 257], [700, 3]])
def test_cache_against_softmax(lengths):
    rng = np.random.default_rng(len(lengths))
    heads, kv, d, n = 4, 2, 16, len(lengths)
    total = sum(lengths) + 5
    cache = dict(k=rng.integers(0, 256, (total, kv, d // 2)).astype(np.uint8), v=rng.integers(0, 256, (total, kv, d // 2)).astype(np.uint8),
                 ke=rng.integers(-4, 0, (total, kv)).astype(np.int8), ve=rng.integers(-4, 2, (total, kv)).astype(np.int8))
    Q = rand_qt(rng, (n, heads * d), o.ROW, -8, -6)
    order, slots, at = rng.permutation(total), [], 0
    for t in lengths:
        slots.append(order[at:at + t])
        at += t
    O = o.attention_cache(Q, cache, slots, heads, kv, d, 0.25)
    for i, row in enumerate(slots):
        for h in range(heads):
            got = values(O)[i, h * d:(h + 1) * d]
            if not len(row):
                assert not got.any()
                continue
            k = np.ldexp(o.unpack4(cache["k"][row, h // 2]).astype(float), cache["ke"][row, h // 2].astype(int)[:, None])
            v = np.ldexp(o.unpack4(cache["v"][row, h // 2]).astype(float), cache["ve"][row, h // 2].astype(int)[:, None])
            t = k @ values(Q)[i, h * d:(h + 1) * d] * 0.25
            p = np.exp(t - t.max())
            L = 32512 * p.sum()
            want = p / p.sum() @ v
            # weights twice (of a key and of its block), numerator and sum, each with its half unit
            vm = 8 * 2.0 ** cache["ve"][row, h // 2].max()
            tol = 4 * W_ERR * (p / p.sum() @ np.abs(v)).max() + 4 * len(row) * 0.5 * vm / L * 1.01
            assert np.all(np.abs(got - want) <= tol + 0.5 * 2.0 ** O.row_exp()[i])
