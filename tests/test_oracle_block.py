"""The oracle of the transformer block's operators (layer norm, the product
with bias, ReLU and residual, the bias gradient, dropout) against closed
forms in exact rationals or 60 digits, against differences, and against
published values of the generator."""

from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np
import pytest

import oracle as o

getcontext().prec = 60
T, R = o.TENSOR, o.ROW


def _dec(v: Fraction) -> Decimal:
    return Decimal(v.numerator) / Decimal(v.denominator)


def _rand(rng, rows, cols, group, elo=-9, ehi=-4):
    n = rows if group == R else 1
    return o.QT(rng.integers(-127, 128, (rows, cols)).astype(np.int8), rng.integers(elo, ehi + 1, n).astype(np.int8),
                group)


def _vec(rng, n, kind, mean=0.0):
    """[n x 1] with one exponent per channel (R) or one (T); [1 x n] for "1"."""
    m = np.clip(np.rint(100 * mean + 25 * rng.normal(size=(n, 1))), -127, 127).astype(np.int8)
    if kind == "1":
        return o.QT(m.reshape(1, n), np.array([-7], np.int8), R)
    return o.QT(m, rng.integers(-8, -5, n if kind == R else 1).astype(np.int8), kind)


def _vals(t):
    return [_dec(v) for row in t.values() for v in row]


def _norm_rows(X, eps):
    """Exact rows and 1 / sigma, in 60 digits."""
    out = []
    for row in X.values():
        n = len(row)
        mean = sum(row) / n
        var = sum((v - mean) ** 2 for v in row) / n
        out.append(([_dec(v - mean) for v in row], 1 / _dec(var + eps.value()).sqrt()))
    return out


def _check_rounded(got: o.QT, want, slack, what):
    """got is want rounded: within half a unit of its exponent plus `slack`
    (per row), and no smaller exponent would hold it."""
    rows = got.mant.shape[0]
    for i in range(rows):
        u = Decimal(2) ** int(got.row_exp()[i])
        for c, v in zip(got.mant[i].reshape(-1), want[i]):
            assert abs(Decimal(int(c)) * u - v) <= u / 2 + slack[i], what
    groups = [list(range(rows))] if got.group == T else [[i] for i in range(rows)]
    for gr in groups:
        top = max(abs(v) for i in gr for v in want[i])
        u = Decimal(2) ** int(got.row_exp()[gr[0]])
        if int(got.row_exp()[gr[0]]) > o.E_MIN:
            assert top + max(slack[i] for i in gr) >= u / 2 * (Decimal(2 * 127 + 1) / 2), what + ": exponent too large"


@pytest.mark.parametrize("n", [2, 3, 17, 64])
@pytest.mark.parametrize("groups", [(T, T), (R, R), (R, T)], ids=["TT", "RR", "RT"])
@pytest.mark.parametrize("kind", [None, T, R, "1"], ids=["none", "T", "R", "1xN"])
def test_layer_norm_fwd(n, groups, kind):
    rng = np.random.default_rng(n + 10 * groups[0])
    X = _rand(rng, 4, n, groups[0])
    g, b = (None, None) if kind is None else (_vec(rng, n, kind, 1.0), _vec(rng, n, kind))
    eps = o.Scalar(85, -23)
    Y = o.layer_norm_fwd(X, g, b, eps, groups[1])
    gv = [Decimal(1)] * n if g is None else _vals(g)
    bv = [Decimal(0)] * n if b is None else _vals(b)
    want = [[d * r * gj + bj for d, gj, bj in zip(dev, gv, bv)] for dev, r in _norm_rows(X, eps)]
    # t, its root, the quotient, h and h gamma each round by 2^-53, the sum by 2^-53 of itself
    slack = [max(abs(d * r * gj) + abs(bj) for d, gj, bj in zip(dev, gv, bv)) * 8 / Decimal(2) ** 53
             for dev, r in _norm_rows(X, eps)]
    _check_rounded(Y, want, slack, f"n={n}")


def test_layer_norm_flat_rows():
    """Rows without deviations give beta, with eps = 0 too; the widths."""
    X = o.QT(np.array([[5, 5, 5], [0, 0, 0], [-128, -128, -128]], np.int8), np.array([-3, -128, 100], np.int8), R)
    b = o.QT(np.array([[64], [-32], [1]], np.int8), np.array([-6], np.int8), T)
    for eps in (o.Scalar(0, 0), o.Scalar(1, -20)):
        Y = o.layer_norm_fwd(X, None, b, eps, R)
        assert np.array_equal(Y.mant, np.array([[64, -32, 1]] * 3)) and np.all(Y.exp == -6)
        assert np.all(o.layer_norm_fwd(X, None, None, eps, R).exp == o.E_MIN)
        dX, dg, db = o.layer_norm_bwd(X, X, None, eps, R, T)
        assert not dX.mant.any() and not dg.mant.any()
    Y4 = o.layer_norm_fwd(X, None, b, o.Scalar(0, 0), R, bits=4)
    assert np.abs(Y4.mant).max() <= 7


def _dx_real(dy, gv, dev, r):
    n = len(dev)
    g = [a * b for a, b in zip(dy, gv)]
    h = [d * r for d in dev]
    m1, m2 = sum(g) / n, sum(a * b for a, b in zip(g, h)) / n
    return [r * (a - m1 - b * m2) for a, b in zip(g, h)], g, h


@pytest.mark.parametrize("n", [2, 5, 33])
@pytest.mark.parametrize("groups", [(T, T, T), (R, T, R), (R, R, R)], ids=["TTT", "RTR", "RRR"])
def test_layer_norm_bwd(n, groups):
    """dX, dgamma and dbeta against the formula, gamma with one exponent (so
    that nothing is lost by re-expressing it)."""
    rng = np.random.default_rng(n)
    X, dY = _rand(rng, 6, n, groups[0]), _rand(rng, 6, n, groups[1], -14, -9)
    gam = _vec(rng, n, T, 1.0)
    eps = o.Scalar(85, -23)
    dX, dg, db = o.layer_norm_bwd(dY, X, gam, eps, groups[2], R)
    gv = _vals(gam)
    rows = _norm_rows(X, eps)
    dyv = [[_dec(v) for v in row] for row in dY.values()]
    want, slack, hs = [], [], []
    for dy, (dev, r) in zip(dyv, rows):
        w, g, h = _dx_real(dy, gv, dev, r)
        want.append(w)
        hs.append(h)
        # f is h off by at most 2^-21: once in sum g f, once in f itself
        s1, s2 = sum(abs(a) for a in g) / n, abs(sum(a * b for a, b in zip(g, h))) / n
        slack.append(r * (max(abs(v) for v in h) * s1 + s2 + s1) / Decimal(2) ** 20)
    _check_rounded(dX, want, slack, f"dX n={n}")
    a, e = o.align_rows(dY)
    av = [[Decimal(int(v)) * Decimal(2) ** int(e) for v in row] for row in a]
    for j in range(n):
        for name, got, ref, sl in (
                ("dgamma", dg, sum(av[i][j] * hs[i][j] for i in range(6)),
                 sum(abs(av[i][j]) for i in range(6)) / Decimal(2) ** 21),
                ("dbeta", db, sum(av[i][j] for i in range(6)), Decimal(0))):
            u = Decimal(2) ** int(got.exp[j])
            assert abs(Decimal(int(got.mant[j, 0])) * u - ref) <= u / 2 + sl, name


def test_layer_norm_bwd_against_differences():
    """dX against central differences of sum dY . y in 60 digits."""
    rng = np.random.default_rng(3)
    n, eps = 9, o.Scalar(85, -23)
    X, dY, gam = _rand(rng, 2, n, T), _rand(rng, 2, n, T, -10, -10), _vec(rng, n, T, 1.0)
    dX, _, _ = o.layer_norm_bwd(dY, X, gam, eps, R, T)
    gv, dyv = _vals(gam), [[_dec(v) for v in row] for row in dY.values()]
    xs = [[_dec(v) for v in row] for row in X.values()]

    def loss(row, dy):
        mean = sum(row) / n
        r = 1 / (sum((v - mean) ** 2 for v in row) / n + _dec(eps.value())).sqrt()
        return sum(a * (v - mean) * r * g for a, v, g in zip(dy, row, gv))

    step = Decimal(10) ** -15
    for i in range(2):
        u = Decimal(2) ** int(dX.exp[i])
        for j in range(n):
            up, dn = list(xs[i]), list(xs[i])
            up[j] += step
            dn[j] -= step
            num = (loss(up, dyv[i]) - loss(dn, dyv[i])) / (2 * step)
            # half a unit for the rounding, 2^-10 of one for f's 2^-21 (as above) and the difference's own error
            assert abs(Decimal(int(dX.mant[i, j])) * u - num) <= u * (Decimal(1) / 2 + Decimal(2) ** -10)


@pytest.mark.parametrize("group", [T, R])
def test_bias_gradient(group):
    rng = np.random.default_rng(5)
    dY = _rand(rng, 11, 7, group)
    a, e = o.align_rows(dY)
    for vg in (T, R):
        got = o.linear_bwd_db(dY, vg)
        ref, exps = o.requant_frac([[Fraction(int(v)) * Fraction(2) ** int(e)] for v in a.sum(axis=0)], vg)
        assert got.mant.tolist() == ref and got.exp.tolist() == exps
    assert not o.linear_bwd_db(o.QT(np.zeros((0, 3), np.int8), np.array([4], np.int8), T), R).mant.any()


@pytest.mark.parametrize("groups", [(T, T, T, T, T), (R, R, R, R, R), (R, T, R, T, R), (T, R, T, R, T)],
                         ids=["T", "R", "RTRTR", "TRTRT"])
@pytest.mark.parametrize("bits", [8, 5])
def test_linear_fused_is_the_exact_sum(groups, bits):
    """While the three terms span at most 53 bits the result is the exact sum
    rounded once; without bias and residual it is the plain product."""
    rng = np.random.default_rng(7)
    X, W = _rand(rng, 5, 12, groups[0]), _rand(rng, 6, 12, groups[1])
    b, D = _vec(rng, 6, groups[2]), _rand(rng, 5, 6, groups[3])
    got = o.linear_fwd_fused(X, W, b, D, groups[4], bits=bits)
    acc, eps = o.linear_fwd_acc(X, W)
    bv = [v for row in b.values() for v in row]
    vals = [[Fraction(int(acc[i, j])) * Fraction(2) ** int(eps[i, j]) + bv[j] + D.values()[i][j] for j in range(6)]
            for i in range(5)]
    ref, exps = o.requant_frac(vals, groups[4], bits)
    assert got.mant.tolist() == ref and got.exp.tolist() == exps
    plain = o.linear_fwd_fused(X, W, None, None, groups[4], bits=bits)
    want = o.linear_fwd(X, W, groups[4], bits)
    assert np.array_equal(plain.mant, want.mant) and np.array_equal(plain.exp, want.exp)
    clipped = o.linear_fwd_fused(X, W, b, D, groups[4], relu=True, bits=bits)
    assert np.array_equal(clipped.mant, np.maximum(got.mant, 0)) and np.array_equal(clipped.exp, got.exp)


def test_philox_published_values():
    """Known answers of Philox4x32 with 10 rounds."""
    f = 0xFFFFFFFF
    assert o.philox4x32((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert o.philox4x32((f, f, f, f), (f, f)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert o.philox4x32((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_dropout():
    rng = np.random.default_rng(9)
    X, D = _rand(rng, 6, 37, R), _rand(rng, 6, 37, T)
    for drop in (0, 6554, 32768, 65535):
        keep = o.dropout_draws(6, 37, 1234567890123456789, 7) >= drop
        scale = Fraction(float(np.float32(65536 / (65536 - drop))))
        assert abs(scale * (65536 - drop) / 65536 - 1) <= Fraction(1, 1 << 24)
        for res in (None, D):
            got = o.dropout(X, res, drop, 1234567890123456789, 7, R)
            vals = [[(v * scale if keep[i, j] else Fraction(0)) + (res.values()[i][j] if res else 0)
                     for j, v in enumerate(row)] for i, row in enumerate(X.values())]
            ref, exps = o.requant_frac(vals, R)
            assert got.mant.tolist() == ref and got.exp.tolist() == exps
    # drop = 0 keeps everything, one half only moves the exponent
    same = o.dropout(X, None, 0, 1, 2, R)
    assert np.array_equal(np.ldexp(same.mant.astype(float), same.exp[:, None]),
                          np.ldexp(X.mant.astype(float), X.exp[:, None]))


def test_dropout_draws_are_uniform_and_apart():
    """The draws of 40 x 4096 elements: their mean, the share below a
    threshold, neighbours and steps uncorrelated (five standard deviations)."""
    u = np.concatenate([o.dropout_draws(10, 2048, 99, s) for s in (0, 1, 1 << 33)])
    n = u.size
    assert abs(u.mean() - 32767.5) < 5 * 65536 / np.sqrt(12 * n)
    assert abs((u < 6554).mean() - 0.1) < 5 * np.sqrt(0.09 / n)
    v = (u - u.mean()) / u.std()
    for a, b in ((v[:, 1:], v[:, :-1]), (v[1:], v[:-1]), (v[10:20], v[:10]), (v[20:], v[:10])):
        assert abs((a * b).mean()) < 5 / np.sqrt(a.size)
