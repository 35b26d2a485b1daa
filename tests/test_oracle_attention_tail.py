"""The oracle's attention where most of softmax's weight, or all of its result, lies in thousands of small weights, against
softmax in 64 bits."""

import numpy as np
import pytest

import oracle as o
from tests.attention_tail import marks, sink
from tests.test_oracle_attention import W_ERR, softmax64, values

# nats that the sink is ahead, exponent of its row above the others', mean of the other values
SINKS = [(3000, 9.4, 2, 0.0), (3000, 10.6, 0, 0.0), (3000, 10.6, 0, 30.0), (3000, 12.0, 2, 10.0), (4096, 11.0, 4, 0.0)]


def forward_tolerance(X, p, v, L, fine, e):
    """How far a head's o may be from softmax's, [rows]: weights off by W_ERR relative twice (numerator and sum), and by half a
    unit each in both sums, a unit being 2^-14 in rows of fine weights."""
    n, unit = p.shape[1], np.where(fine, 2.0 ** -o.ATT_FINE, 1.0)
    rate = 2 * W_ERR * (p @ np.abs(v)).max(axis=1)
    return rate + n * (127 * 2.0 ** e.max() + np.abs(v).max()) * 0.5 * unit / L


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("n,gap,lift,mean", SINKS)
def test_forward_keeps_the_tail(n, gap, lift, mean, causal):
    rng = np.random.default_rng(int(10 * gap) + lift)
    X, scale = sink(rng, n, gap, lift=lift, mean=mean)
    O, tops, sums = o.attention_fwd(X, 1, 1, 16, scale, causal, [0, n])
    _, want, ps = softmax64(X, 1, 1, 16, scale, causal, [0, n])
    (_, _, p, v, _, _), = ps
    fine = marks(tops)[:, 0]
    assert fine[o.ATT_CHECK:].all() and not fine[:o.ATT_CHECK if causal else 0].any()
    tol = forward_tolerance(X, p[0], v[0], sums[:, 0].astype(np.float64), fine, X.row_exp()) + 0.5 * np.ldexp(1.0, O.row_exp())
    err = np.abs(values(O) - want.detach().numpy()).max(axis=1)
    assert np.all(err <= tol)
    # and of the tail's rows little is lost: the tolerance itself is a small part of the result, half a unit of its rounding (1 / 128)
    # and the half units of fine weights, at most 3000 * 127 (2^2 + 1) / 2^15 / 33050 = 0.0018 of 2^e on results of 0.137 and more
    # (with a lift of 4 they may come to 4096 * 127 (2^4 + 1) / 2^15 / 34659 = 0.0078, on results of 0.05: a bound that says little)
    size = np.abs(want.detach().numpy()).max(axis=1)
    assert lift == 4 or np.median((tol / size)[o.ATT_CHECK:]) < 1 / 128 + 0.0018 / 0.137


def test_tensor_group_and_flat_rows():
    """One exponent for all tokens; rows that see the sink among rows of equal weights, which keep their integers."""
    rng = np.random.default_rng(3)
    X, scale = sink(rng, 2500, 11.0, group=o.TENSOR, flat_rows=True)
    O, tops, sums = o.attention_fwd(X, 1, 1, 16, scale, False, [0, 2500])
    _, want, ((_, _, p, v, _, _),) = softmax64(X, 1, 1, 16, scale, False, [0, 2500])
    fine = marks(tops)[:, 0]
    assert fine[0::2].all() and not fine[1::2].any()
    tol = forward_tolerance(X, p[0], v[0], sums[:, 0].astype(np.float64), fine, X.row_exp()) + 0.5 * np.ldexp(1.0, O.row_exp())
    assert np.all(np.abs(values(O) - want.detach().numpy()).max(axis=1) <= tol)


def test_rows_of_few_keys_stay_coarse():
    """Up to ATT_CHECK keys a weight has 15 bits: rounding takes at most a 32nd of the sum."""
    assert o.ATT_CHECK / 2 == o.ATT_UNIT / 32
    rng = np.random.default_rng(4)
    X, scale = sink(rng, o.ATT_CHECK, 10.6)
    _, tops, sums = o.attention_fwd(X, 1, 1, 16, scale, False)
    assert not marks(tops).any()
    t = (X.mant[:, :16].astype(float) @ X.mant[:, 16:32].astype(float).T) * 2.0 ** (2 * int(X.exp[0])) * scale
    den = np.exp(t - t.max(axis=1, keepdims=True)).sum(axis=1) * o.ATT_UNIT
    assert np.all(np.abs(sums[:, 0] - den) <= den * (W_ERR + 1e-5) + o.ATT_UNIT / 32)
