"""Outputs of the block operators that lie partly over an input, or over
another output, are refused on the host; ones that only touch it are not (the
call then gets as far as its missing workspace)."""

import ctypes

import pytest

from integer_only_dnn_amd import ie

by = ctypes.byref
BIG = 1 << 30
WORKSPACE, UNSUPPORTED = 4, 6
# rows, cols, mantissas' and exponents' first byte of operands far from each other
A, B = 1 << 16, 1 << 20


def mat(rows, cols, mant, exp, group=1):
    return ie.ie_mat(mant, exp, rows, cols, group, 0)


# where an output of 16 x 32 mantissas and 16 exponents lies beside an operand
# of the same size with mantissas at A and exponents at A + 4096
PLACES = [("one row down", A + 32, B, UNSUPPORTED), ("last byte", A + 511, B, UNSUPPORTED),
          ("first byte", A - 511, B, UNSUPPORTED), ("behind", A + 512, B, WORKSPACE), ("before", A - 512, B, WORKSPACE),
          ("exponents one row down", B, A + 4097, UNSUPPORTED), ("exponents behind", B, A + 4112, WORKSPACE),
          ("exponents in the mantissas", B, A + 500, UNSUPPORTED),
          ("mantissas over the exponents", A + 4096 - 8, B, UNSUPPORTED),
          ("mantissas up to the exponents", A + 4096 - 512, B, WORKSPACE)]


@pytest.mark.parametrize("what,m,e,want", PLACES, ids=[p[0] for p in PLACES])
def test_overlapping_outputs(what, m, e, want):
    L = ie.lib()
    X, Y = mat(16, 32, A, A + 4096), mat(16, 32, m, e)
    far, eps = mat(16, 32, 1 << 24, 1 << 25), ie.ie_scalar(85, -23)
    d = ie.ie_dropout_desc(1, 2, None, 6554)
    assert L.ie_layer_norm_fwd(by(X), None, None, eps, by(Y), None, BIG, None) == want
    assert L.ie_layer_norm_bwd(by(X), by(far), None, eps, by(Y), None, None, None, BIG, None) == want
    assert L.ie_layer_norm_bwd(by(far), by(X), None, eps, by(Y), None, None, None, BIG, None) == want
    assert L.ie_dropout(by(X), None, by(Y), by(d), None, BIG, None) == want
    assert L.ie_dropout(by(far), by(X), by(Y), by(d), None, BIG, None) == want
    # [16 x 32] = [16 x 64] . [32 x 64]^T + X; the same as an input and as a weight
    x, w = mat(16, 64, 1 << 21, 1 << 22), mat(32, 64, 1 << 23, 1 << 26)
    assert L.ie_linear_fwd_fused(by(x), by(w), None, by(X), by(Y), 0, None, BIG, None) == want
    sq = mat(32, 32, 1 << 23, 1 << 26)
    assert L.ie_linear_fwd_fused(by(X), by(sq), None, None, by(Y), 0, None, BIG, None) == want


def test_overlapping_plain_products():
    """The product without addends by the dense tiles: 2000 x 64 over its input or its weight."""
    L = ie.lib()
    X, W = mat(2000, 64, 1 << 24, 1 << 25), mat(64, 64, 1 << 22, 1 << 23)
    for m, e, want in (((1 << 24) + 64, B, UNSUPPORTED), ((1 << 22) + 4095, B, UNSUPPORTED),
                       ((1 << 24) + 2000 * 64, B, WORKSPACE), ((1 << 22) + 4096, B, WORKSPACE),
                       (1 << 26, (1 << 25) + 1999, UNSUPPORTED), (1 << 26, (1 << 25) + 2000, WORKSPACE)):
        got = L.ie_linear_fwd_fused(by(X), by(W), None, None, by(mat(2000, 64, m, e)), 0, None, BIG, None)
        assert got == want, (m, e)


def test_overlapping_vectors():
    """Parameter vectors: 32 channels beside each other, the input and gamma."""
    L = ie.lib()
    X, dY, eps = mat(16, 32, A, A + 4096), mat(16, 32, 1 << 24, 1 << 25), ie.ie_scalar(85, -23)
    dX, gam = mat(16, 32, 1 << 26, 1 << 27), mat(32, 1, B, B + 64)
    for m, e, want in ((B + 31, B + 512, UNSUPPORTED), (B + 32, B + 512, WORKSPACE), (B + 512, B + 95, UNSUPPORTED),
                       (B + 512, B + 96, WORKSPACE), (B + 512, B + 16, UNSUPPORTED), (A + 511, B + 512, UNSUPPORTED),
                       ((1 << 26) + 511, B + 512, UNSUPPORTED), ((1 << 26) + 512, B + 512, WORKSPACE)):
        v = mat(32, 1, m, e)
        assert L.ie_layer_norm_bwd(by(dY), by(X), by(gam), eps, by(dX), by(v), None, None, BIG, None) == want, (m, e)
        assert L.ie_layer_norm_bwd(by(dY), by(X), by(gam), eps, by(dX), None, by(v), None, BIG, None) == want, (m, e)
    g, b = mat(32, 1, B + 512, B + 1024), mat(32, 1, B + 543, B + 2048)
    assert L.ie_layer_norm_bwd(by(dY), by(X), by(gam), eps, by(dX), by(g), by(b), None, BIG, None) == UNSUPPORTED
    # one exponent for the vector takes one byte, one per channel 32
    for group, want in ((0, WORKSPACE), (1, UNSUPPORTED)):
        v = mat(32, 1, B + 512, (1 << 25) - 1, group)
        assert L.ie_linear_bwd_db(by(dY), by(v), None, BIG, None) == want
    assert L.ie_linear_bwd_db(by(dY), by(mat(32, 1, (1 << 24) + 500, B)), None, BIG, None) == UNSUPPORTED
