"""What layer norm's backward pass loses by re-expressing gamma at its largest
channel exponent: the input gradient of the oracle against the formula with
the exact gamma."""

from decimal import Decimal

import numpy as np
import pytest

import oracle as o
from tests.test_oracle_block import _check_rounded, _dec, _dx_real, _norm_rows, _rand, _vals

R, T = o.ROW, o.TENSOR
EPS = o.Scalar(85, -23)


@pytest.mark.parametrize("spread", [0, 1, 3, 7, 8, 20])
@pytest.mark.parametrize("n", [5, 40])
def test_error_of_dx_is_half_a_unit_of_gammas_largest_exponent(n, spread):
    """gamma' = gamma + d with |d| <= 2^(top - 1), and dX is linear in gamma, so that beside its own rounding
    and that of h (2^-20, see test_layer_norm_bwd) dX_j is off by at most
    r 2^(top - 1) (|dY_j| + mean |dY| + |h_j| mean |dY h|)."""
    rng = np.random.default_rng(100 * n + spread)
    X, dY = _rand(rng, 6, n, R), _rand(rng, 6, n, R, -14, -9)
    gam = o.QT(rng.integers(-127, 128, (n, 1)).astype(np.int8), rng.integers(-7 - spread, -6, n).astype(np.int8), R)
    dX, _, _ = o.layer_norm_bwd(dY, X, gam, EPS, R, R)
    half = Decimal(2) ** (int(gam.exp.max()) - 1)
    dyv, gv = [[_dec(v) for v in row] for row in dY.values()], _vals(gam)
    want, slack = [], []
    for dy, (dev, r) in zip(dyv, _norm_rows(X, EPS)):
        w, g, h = _dx_real(dy, gv, dev, r)
        want.append(w)
        size = [abs(a) for a in dy]
        far = [abs(a * b) for a, b in zip(dy, h)]
        lost = half * (max(size) + sum(size) / n + max(abs(v) for v in h) * sum(far) / n)
        big = [abs(a) + half * b for a, b in zip(g, size)]
        top = max(abs(v) for v in h)
        of_f = (top * sum(big) / n + sum(abs(v) * b for v, b in zip(h, big)) / n + sum(big) / n) / Decimal(2) ** 20
        slack.append(r * (lost * (1 if spread else 0) + of_f))
    _check_rounded(dX, want, slack, f"spread {spread}")


@pytest.mark.parametrize("below", [7, 8, 9, 60])
def test_channels_eight_exponents_below_count_as_zero(below):
    """A mantissa of at most 128 at 8 places below rounds to 0 (a tie at most, and 0 is even); at 7 it is still 1."""
    rng = np.random.default_rng(below)
    X, dY = _rand(rng, 3, 12, R), _rand(rng, 3, 12, R, -14, -9)
    gam = o.QT(np.full((12, 1), -128, np.int8), np.full(12, -7, np.int8), R)
    gam.exp[4:] = -7 - below
    none = o.QT(np.where(np.arange(12)[:, None] < 4, gam.mant, 0).astype(np.int8), np.full(12, -7, np.int8), R)
    got, zero = o.layer_norm_bwd(dY, X, gam, EPS, R, R), o.layer_norm_bwd(dY, X, none, EPS, R, R)
    same = np.array_equal(got[0].mant, zero[0].mant) and np.array_equal(got[0].exp, zero[0].exp)
    assert same == (below >= 8)
    # the gradients of gamma and beta do not depend on gamma
    for a, b in zip(got[1:], zero[1:]):
        assert np.array_equal(a.mant, b.mant) and np.array_equal(a.exp, b.exp)
