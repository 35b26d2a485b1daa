"""The oracle's attention where most of softmax's weight, or all of its result, lies in thousands of small weights, against
softmax in 64 bits."""

import numpy as np
import pytest
import torch

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


def backward_tolerances(X, O, dO, o64, p, v, k, q, L, fine, scale, d):
    """Elementwise bounds of the errors of dQ, dK, dV of one head over one sequence, before the last rounding: weights off by W_ERR
    relative twice and by half a unit of L (and by its rounding to whole units), D from the rounded O, fp32 roundings, and half a
    unit of every integer that enters a sum."""
    n, small = p.shape[0], 2.0 ** -o.ATT_FINE
    e, ed = X.row_exp(), dO.row_exp()
    dy, unit = values(dO), np.where(fine, small, 1.0)
    dD = (np.abs(dy) * np.abs(values(O) - o64)).sum(axis=1)
    dP = dy @ v.T
    mean = (p * dP).sum(axis=1, keepdims=True)
    big = np.abs(dP) + np.abs(mean)
    perr = p * (2 * W_ERR + (0.5 * n * unit / L)[:, None] + (0.5 / L)[:, None] + 2.0 ** -22)
    serr = perr * big + (p + perr) * (dD[:, None] + 2.0 ** -22 * big)
    dq, dk, dv = scale * serr @ np.abs(k), scale * serr.T @ np.abs(q), perr.T @ np.abs(dy)
    # the integers' scales: powers of two at most 2^2 times the norms' products they stand for
    vn, dn = 2 * np.linalg.norm(v, axis=1).max(), 2 * np.linalg.norm(dy, axis=1)
    dot = 2 * np.abs((dy * values(O)).sum(axis=1))
    top = 2 * np.maximum(dn * vn, dot) * 127 * np.ldexp(1.0, int(e.max()))
    dq += (scale * 0.5 * top * unit * n / L)[:, None]
    am = (2.0 ** np.maximum(ed - ed.max(), -60) / L).max() * 2 * 2.0 ** ed.max()
    dv += 0.5 * am * small * np.abs(dO.mant.astype(np.float64)).max() * n
    lm = (2.0 ** np.maximum(ed - ed.max(), -60) / L * 4 * np.maximum(dn / 2.0 ** ed * vn, dot / 2.0 ** ed) * 2.0 ** e).max() * 2.0 ** ed.max()
    dk += scale * 0.5 * lm * small * 127 * n
    return dq, dk, dv


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("n,gap,lift,mean", [(3000, 10.6, 0, 0.0), (2600, 10.5, 2, 0.0), (2600, 12.0, 0, 20.0)])
def test_gradient_keeps_the_tail(n, gap, lift, mean, causal):
    rng = np.random.default_rng(int(10 * gap) + lift)
    X, scale = sink(rng, n, gap, lift=lift, mean=mean)
    O, tops, sums = o.attention_fwd(X, 1, 1, 16, scale, causal, [0, n])
    dO = o.QT(np.clip(np.rint(rng.normal(10, 40, (n, 16))), -127, 127).astype(np.int8), rng.integers(-16, -13, n).astype(np.int8), o.ROW)
    G = values(o.attention_bwd(X, O, dO, tops, sums, 1, 1, 16, scale, causal, [0, n]))
    x, y, ((_, _, p, v, k, q),) = softmax64(X, 1, 1, 16, scale, causal, [0, n])
    want = torch.autograd.grad((y * torch.from_numpy(values(dO))).sum(), x)[0].numpy()
    tol = np.concatenate(backward_tolerances(X, O, dO, y.detach().numpy(), p[0], v[0], k[0], q[0], sums[:, 0].astype(np.float64),
                                             marks(tops)[:, 0], scale, 16), axis=1)
    half = 0.5 * np.ldexp(1.0, o.requant_f64(G, o.ROW).row_exp())[:, None]
    assert np.all(np.abs(G - want) <= tol + half)
    # most of a token's dV is not rounding: with one digit less it is nothing at all
    size = np.abs(want[:, 32:]).max(axis=1)
    assert np.median((tol[:, 32:].max(axis=1) / size)[1:o.ATT_CHECK]) < 0.25
