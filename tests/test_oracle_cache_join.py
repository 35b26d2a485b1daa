"""Joining the blocks of a cache: exact sums, whatever their size and order."""

import numpy as np
import pytest

import oracle as o
from tests.test_oracle_attention import W_ERR


def test_sums_of_the_largest_caches_are_exact():
    """2^23 positions, all weights near one, values of 7 and -8: sums of up to 2^55.9, where float64 rounds."""
    rng = np.random.default_rng(1)
    blocks, d = 1 << 15, 4
    lb = rng.integers(250 * 32512, 256 * 32512 + 1, blocks)
    nb = rng.choice([7, -8], (blocks, 1)) * lb[:, None] - rng.integers(0, 9, (blocks, d))
    nb[:, 1], nb[:, 2] = np.abs(nb[:, 1]), -np.abs(nb[:, 2])
    m = -rng.integers(0, 300, blocks) * 2.0 ** -12
    total, num = o.cache_sums([(m[b], lb[b], 0, nb[b].astype(np.float64)) for b in range(blocks)], np.float64(1.0))[:2]
    w = [int(x) for x in np.rint(o.softmax_weight(o.ie_oracle._f32(m - m.max()), np.float64(1.0)))]
    assert int(total) == sum(a * int(b) for a, b in zip(w, lb))
    want = [sum(a * int(b) for a, b in zip(w, nb[:, k])) for k in range(d)]
    assert max(abs(x) for x in want) > 1 << 55
    assert [int(x) for x in num] == want
    # in float64, as rounded sums, they differ from it and from one order to another
    floats = np.cumsum(np.array(w, float)[:, None] * nb, axis=0)[-1]
    assert any(int(f) != x for f, x in zip(floats, want))


def sink_cache(rng, n, gap, d=16, mean=0, ahead=0):
    """(cache, Q, scale): key `ahead` is `gap` nats in front of n - 1 others, and its value is zero."""
    k, v = np.zeros((n, 1, d), np.int64), np.clip(np.rint(rng.normal(mean, 3, (n, 1, d))), -7, 7)
    k[:, :, 1:] = rng.integers(-1, 2, (n, 1, d - 1))
    k[ahead], v[ahead] = 0, 0
    k[ahead, 0, 0] = 7
    ke = np.full((n, 1), -6)
    ke[ahead] = 0
    ve = np.where(v.any(axis=2), -2, -128)
    cache = dict(k=o.pack4(k), v=o.pack4(v), ke=ke.astype(np.int8), ve=ve.astype(np.int8))
    Q = np.zeros((1, d), np.int64)
    Q[0, 0] = 100
    Q[0, 1:] = rng.integers(-60, 61, d - 1)
    return cache, o.QT(Q.astype(np.int8), np.array([-8], np.int8), o.ROW), gap / (7 * 100 / 256)


@pytest.mark.parametrize("n,gap,mean", [(4000, 10.5, 0), (131072, 12.0, 1), (131072, 12.0, 0), (131072, 13.5, 2), (300000, 11.5, 1)])
def test_a_long_tail_is_kept(n, gap, mean):
    """Against softmax in 64 bits.  Errors: weights off by W_ERR relative, of a key and of its block, in numerator and sum;
    half a unit of a key's weight under its block's; half a unit of 2^-14 of a block's."""
    rng = np.random.default_rng(n)
    cache, Q, scale = sink_cache(rng, n, gap, mean=mean)
    O = o.attention_cache(Q, cache, [np.arange(n)], 1, 1, 16, scale)
    k = np.ldexp(o.unpack4(cache["k"][:, 0]).astype(float), cache["ke"].astype(int))
    v = np.ldexp(o.unpack4(cache["v"][:, 0]).astype(float), cache["ve"].astype(int))
    t = k @ (Q.mant[0].astype(float) / 256) * float(np.float32(scale))
    p = np.exp(t - t.max())
    want = p / p.sum() @ v
    at = np.arange(0, n, 256)
    m, size = np.maximum.reduceat(p, at), np.add.reduceat(p, at)
    vm = 7 * 2.0 ** -2
    tol = 4 * W_ERR * (p / p.sum() @ np.abs(v)).max() + 2 * (m * 128 / 32512).sum() / p.sum() * vm
    tol += 2 * (0.5 * 2.0 ** -14 / 32512 * size / m).sum() / p.sum() * vm
    got = O.mant[0].astype(float) * 2.0 ** int(O.exp[0])
    assert np.all(np.abs(got - want) <= tol + 0.5 * 2.0 ** int(O.exp[0]))
    # coarse weights give zeros, or lose most of it; values about zero cancel, and the bound does not
    assert mean == 0 or tol < 0.5 * np.abs(want).max()


def test_few_blocks_stay_coarse():
    """Blocks of weights just below half a unit: up to CACHE_CHECK of them are left out, which is less than a 32nd; more are not."""
    for n in (o.CACHE_CHECK, 40):
        parts = [(0.0, 32512, 0, np.full(16, 32512.0))] + (n - 1) * [(-16.1, 256 * 32512, 0, np.full(16, 2.0 * 256 * 32512))]
        got, s = o.cache_join(parts, np.float64(1.0), n), (n - 1) * 256 * 2.0 ** -16.1
        if n == o.CACHE_CHECK:
            assert s < 1 / 32 and np.allclose(got, 1.0, rtol=1e-15)
        else:  # a weight's error and half a unit of 2^-14 of 0.46
            assert np.allclose(got, (1 + 2 * s) / (1 + s), rtol=W_ERR + 0.5 * 2.0 ** -14 / 0.46)


def test_a_small_tail_that_is_the_whole_result():
    """A tail of a 45th of the weight, beside a key whose value is zero: the weights' sum hardly changes, the values' is all there
    is.  Tolerances as above, a key's rounding taking no more than its weight."""
    rng, n = np.random.default_rng(8), 131072
    cache, Q, scale = sink_cache(rng, n, 15.6, mean=2)
    O = o.attention_cache(Q, cache, [np.arange(n)], 1, 1, 16, scale)
    k = np.ldexp(o.unpack4(cache["k"][:, 0]).astype(float), cache["ke"].astype(int))
    v = np.ldexp(o.unpack4(cache["v"][:, 0]).astype(float), cache["ve"].astype(int))
    t = k @ (Q.mant[0].astype(float) / 256) * float(np.float32(scale))
    p = np.exp(t - t.max())
    want = p / p.sum() @ v
    assert 0.01 < (p.sum() - 1) / p.sum() < 1 / 32
    at = np.arange(0, n, 256)
    m, size = np.maximum.reduceat(p, at), np.add.reduceat(p, at)
    vm = 7 * 2.0 ** -2
    tol = 4 * W_ERR * (p / p.sum() @ np.abs(v)).max() + 2 * np.minimum(m.repeat(256) * 0.5 / 32512, p).sum() / p.sum() * vm
    tol += 2 * (0.5 * 2.0 ** -14 / 32512 * size / m).sum() / p.sum() * vm
    assert np.all(np.abs(O.mant[0] * 2.0 ** int(O.exp[0]) - want) <= tol + 0.5 * 2.0 ** int(O.exp[0]))
    assert tol < 0.5 * np.abs(want).max()
