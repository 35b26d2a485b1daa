"""The oracle's attention at the ends of the exponents' range, against the values themselves."""

import numpy as np
import pytest

import oracle as o
from tests.test_oracle_attention import softmax64, values


@pytest.mark.parametrize("e", [11, 12, 14, 16])
def test_large_rows_through_the_cache(e):
    """Rows of large exponents become larger ones in 4 bits; attention over one key is its value, up to the 4 bits."""
    X = o.QT(np.full((1, 3 * 16), 127, np.int8), np.array([e], np.int8), o.ROW)
    X.mant[0, 32:] = np.arange(-128, 128, 16)
    cache = dict(k=np.zeros((1, 1, 8), np.uint8), v=np.zeros((1, 1, 8), np.uint8), ke=np.zeros((1, 1), np.int8), ve=np.zeros((1, 1), np.int8))
    o.cache_store(cache, X, 1, 1, 16, [0])
    assert int(cache["ve"][0, 0]) == e + 5 and int(cache["ke"][0, 0]) == e + 5
    O = o.attention_cache(X, cache, [np.array([0])], 1, 1, 16, 0.25)
    want, got = X.mant[0, 32:].astype(float) * 2.0 ** e, O.mant[0].astype(float) * 2.0 ** int(O.exp[0])
    assert np.all(np.abs(got - want) <= 0.5 * 2.0 ** (e + 5) + 0.5 * 2.0 ** int(O.exp[0]))


def test_large_keys_order_the_softmax():
    """Two keys, stored from exponent 16: scores 2^5 apart from what a clipped exponent gives."""
    X = o.QT(np.zeros((2, 3 * 16), np.int8), np.full(2, 16, np.int8), o.ROW)
    X.mant[:, 16], X.mant[:, 17] = 127, [0, 64]  # 4 2^21 and 2 2^21
    X.mant[:, 32] = [64, -64]
    cache = dict(k=np.zeros((2, 1, 8), np.uint8), v=np.zeros((2, 1, 8), np.uint8), ke=np.zeros((2, 1), np.int8), ve=np.zeros((2, 1), np.int8))
    o.cache_store(cache, X, 1, 1, 16, [0, 1])
    Q = o.QT(np.zeros((1, 16), np.int8), np.array([-22], np.int8), o.ROW)
    Q.mant[0, 1] = 4
    k = np.ldexp(o.unpack4(cache["k"][:, 0]).astype(float), cache["ke"].astype(int))
    v = np.ldexp(o.unpack4(cache["v"][:, 0]).astype(float), cache["ve"].astype(int))
    p = np.exp(k @ (Q.mant[0] * 2.0 ** -22) * 0.25)
    assert k[1, 1] > 0 and 2 < p[1] / p[0] < 2.0 ** 8
    want, O = p / p.sum() @ v, o.attention_cache(Q, cache, [np.arange(2)], 1, 1, 16, 0.25)
    # two weights, each off by half a unit of 32512 and 1.2e-4 relative, twice
    tol = 2 * (1.2e-4 + 0.5 / 32512 * 2) * np.abs(v).max() + 0.5 * 2.0 ** int(O.exp[0])
    assert np.all(np.abs(O.mant[0].astype(float) * 2.0 ** int(O.exp[0]) - want) <= tol)


def gradient_errors(X, bits, scale, seed, ed=-20):
    """The gradient's relative errors by row (norms of dQ, dK and dV together) against autograd, heads of 16, one sequence."""
    rng, n = np.random.default_rng(seed), X.mant.shape[0]
    O, tops, sums = o.attention_fwd(X, 1, 1, 16, scale, False, None, bits)
    dO = o.QT(rng.integers(-127, 128, (n, 16)).astype(np.int8), np.full(n, ed, np.int8), o.ROW)
    G = values(o.attention_bwd(X, O, dO, tops, sums, 1, 1, 16, scale, False))
    x, _, ((_, _, p, v, k, q),) = softmax64(X, 1, 1, 16, scale, False, [0, n])
    # the definition with D from the O that the pass has rounded
    dy = values(dO)
    u = dy @ v[0].T - (dy * values(O)).sum(axis=1)[:, None]
    s = p[0] * u
    want = np.concatenate([scale * s @ k[0], scale * s.T @ q[0], p[0].T @ dy], axis=1)
    return O, np.linalg.norm(G - want, axis=0).reshape(3, 16), np.linalg.norm(want, axis=0).reshape(3, 16)


def test_gradient_of_a_narrow_result():
    """O in 2 bits at the largest exponents: its own lie 6 above 16."""
    rng = np.random.default_rng(9)
    X = o.QT(rng.integers(-127, 128, (40, 48)).astype(np.int8), np.full(40, 16, np.int8), o.ROW)
    X.mant[:, 32:] = rng.integers(100, 128, (40, 16))
    O, err, size = gradient_errors(X, 2, 2.0 ** -30, 7)
    assert O.row_exp().min() > 16
    # half a unit of 2^-7 of a row's largest element, which is at most 6 of its root mean square: 0.024; weights of 1.2e-4, twice
    assert np.all(err <= 0.025 * size.max())


@pytest.mark.parametrize("exps", [(-60, -50), (-110, -104), (-126, -119)])
def test_small_rows(exps):
    """Tokens of the smallest exponents: their results and the gradient of their values are as exact as any others'."""
    rng = np.random.default_rng(-exps[0])
    X = o.QT(rng.integers(-127, 128, (50, 48)).astype(np.int8), rng.integers(exps[0], exps[1] + 1, 50).astype(np.int8), o.ROW)
    O, tops, sums = o.attention_fwd(X, 1, 1, 16, 1.0, True)
    x, y, ((_, _, p, v, _, _),) = softmax64(X, 1, 1, 16, 1.0, True, [0, 50])
    # all scores are alike: a weight is 32512, its value's exponent takes half a unit of the largest one's
    tol = 0.5 * 127 * 2.0 ** exps[1] / 32512 + 0.5 * np.ldexp(1.0, O.row_exp())
    assert np.all(np.abs(values(O) - y.detach().numpy()).max(axis=1) <= tol)
    dO = o.QT(rng.integers(-127, 128, (50, 16)).astype(np.int8), np.full(50, -12, np.int8), o.ROW)
    G = values(o.attention_bwd(X, O, dO, tops, sums, 1, 1, 16, 1.0, True))
    want = p[0].T @ values(dO)
    half = 0.5 * np.ldexp(1.0, o.requant_f64(G, o.ROW).row_exp())[:, None]
    # 1 / L in fp32 and half a unit of each of 50 integers of at least 16256 / 50
    assert np.all(np.abs(G[:, 32:] - want) <= half + 127 * 2.0 ** -12 * 50 * 0.5 / 16256)


def test_small_values_in_a_cache():
    rng = np.random.default_rng(4)
    cache = dict(k=rng.integers(0, 256, (300, 1, 8)).astype(np.uint8), v=rng.integers(0, 256, (300, 1, 8)).astype(np.uint8),
                 ke=rng.integers(-100, -60, (300, 1)).astype(np.int8), ve=rng.integers(-66, -60, (300, 1)).astype(np.int8))
    Q = o.QT(rng.integers(-127, 128, (1, 16)).astype(np.int8), np.array([-8], np.int8), o.ROW)
    O = o.attention_cache(Q, cache, [np.arange(300)], 1, 1, 16, 0.25)
    v = np.ldexp(o.unpack4(cache["v"][:, 0]).astype(float), cache["ve"].astype(int))
    assert np.all(np.abs(O.mant[0] * 2.0 ** int(O.exp[0]) - v.mean(axis=0)) <= 0.5 * 8 * 2.0 ** -61 / 32512 + 0.5 * 2.0 ** int(O.exp[0]))
