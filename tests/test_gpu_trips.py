"""GPU parity of layer norm, dropout and the product with bias and residual
where a block takes several rows (or tiles) in turn: every split of rows over
threads that can, the last trip ragged or whole, with one exponent per result
row and with one for the whole result.  tests/test_plan_launch.py checks from
the plans that these shapes leave no such split out."""

import numpy as np
import pytest
import torch

import oracle as o
from integer_only_dnn_amd import ie
from tests.gpu_util import announce, assert_same, qt_to_dev, rand_qt

pytestmark = pytest.mark.gpu

T, R = o.TENSOR, o.ROW
EPS = o.Scalar(85, -23)

# from 4096 rows on 16 to 64 threads share a row; below, and above 2048
# columns, more
NORM = [(33000, 50), (17000, 100), (16500, 190), (16390, 250), (16400, 300), (8200, 500), (8300, 767), (4100, 1000),
        (4200, 1500), (4100, 2001), (4096, 2500), (2100, 100), (2100, 300), (2100, 701), (2051, 1000), (600, 1500),
        (600, 2049), (600, 3500), (1031, 4099), (520, 8000), (515, 8195), (513, 12301), (513, 16384)]
DROPOUT = [(50000, 9), (49200, 70), (49153, 130), (25000, 200), (24600, 260), (12300, 390), (12289, 520), (6200, 777),
           (6150, 1030), (1600, 1540), (1540, 2049), (1537, 4099), (520, 6150), (520, 8200), (513, 16385)]


def name(s):
    return "x".join(map(str, s))


@pytest.fixture(scope="module")
def ws():
    return ie.Workspace("cuda")


@pytest.mark.parametrize("shape", NORM, ids=name)
def test_norm(shape, ws):
    announce(f"norm trips {shape}")
    rows, cols = shape
    rng = np.random.default_rng(rows + cols)
    X, dY = rand_qt(rng, shape, R), rand_qt(rng, shape, R, -20, -9)
    X.mant[rows - 1], X.mant[rows // 2], dY.mant[rows // 3] = 5, 0, 0
    dY.exp[rows - 2] = -3  # one row far above the others: the whole-tensor exponent is its own
    gam, bet = rand_qt(rng, (cols, 1), R, -10, -5), rand_qt(rng, (cols, 1), R, -10, -5)
    e = (EPS.mant, EPS.exp)
    Xd, dYd, gd, bd = (qt_to_dev(t) for t in (X, dY, gam, bet))
    for group in (R, T):
        Y, dX = ie.Mat.empty(rows, cols, group), ie.Mat.empty(rows, cols, group)
        dg, db = ie.Mat.empty(cols, 1, group), ie.Mat.empty(cols, 1, group)
        ie.ie_layer_norm_fwd(Xd, gd, bd, e, Y, ws)
        ie.ie_layer_norm_bwd(dYd, Xd, gd, e, dX, dg, db, ws)
        assert_same(Y, o.layer_norm_fwd(X, gam, bet, EPS, group), f"Y {group}")
        for m, w, what in zip((dX, dg, db), o.layer_norm_bwd(dY, X, gam, EPS, group, group), ("dX", "dgamma", "dbeta")):
            assert_same(m, w, f"{what} {group}")
    assert ws.status() == 0


@pytest.mark.parametrize("shape", DROPOUT, ids=name)
def test_dropout(shape, ws):
    announce(f"dropout trips {shape}")
    rows, cols = shape
    rng = np.random.default_rng(rows + cols)
    X, D = rand_qt(rng, shape, R), rand_qt(rng, shape, R)
    X.exp[rows - 1], D.exp[rows // 2] = 1, 2  # the largest values in the last row, and in one between
    Xd, Dd = qt_to_dev(X), qt_to_dev(D)
    for step, (res, group) in enumerate(((D, R), (None, R), (D, T), (None, T))):
        Y = ie.Mat.empty(rows, cols, group)
        ie.ie_dropout(Xd, Dd if res else None, Y, 13107, 77, step, ws)
        assert_same(Y, o.dropout(X, res, 13107, 77, step, group), f"residual {res is not None} {group}")
    assert ws.status() == 0


# the second pass of round-to-odd results (8, 32 and 64 lanes to a row), rows
# padded to whole runs of 16 bytes, split contractions of more rows than blocks
PRODUCT = [(66000, 40, 48, T, None), (17000, 300, 64, T, None), (8300, 1030, 48, R, None), (17000, 1030, 500, R, None),
           (17000, 1030, 500, T, None), (1100, 60, 300, R, "1,1,2,3"), (1100, 60, 300, T, "1,1,2,3")]


@pytest.mark.parametrize("case", PRODUCT, ids=name)
def test_product(case, ws, monkeypatch):
    announce(f"product trips {case}")
    M, N, K, group, plan = case
    rng = np.random.default_rng(M + N + K)
    X, W = rand_qt(rng, (M, K), R), rand_qt(rng, (N, K), R)
    X.mant[M - 1] = 0
    X.exp[M // 2] = 1
    b, D = rand_qt(rng, (N, 1), R, -12, -5), rand_qt(rng, (M, N), R, -10, 2)
    if plan:
        monkeypatch.setenv("IE_TILE", plan)
    Y = ie.Mat.empty(M, N, group)
    ie.ie_linear_fwd_fused(qt_to_dev(X), qt_to_dev(W), qt_to_dev(b), qt_to_dev(D), Y, ie.ACT_RELU, ws)
    assert_same(Y, o.linear_fwd_fused(X, W, b, D, group, True), str(case))
    assert ws.status() == 0


def test_bias_gradient_of_many_rows(ws):
    """Chunks of several trips each, one shorter than the others."""
    for rows, cols in ((300001, 40), (70000, 700)):
        announce(f"bias gradient trips {rows} x {cols}")
        dY = rand_qt(np.random.default_rng(rows), (rows, cols), R, -20, -9)
        dY.exp[rows - 1] = -5
        for group in (R, T):
            db = ie.Mat.empty(cols, 1, group)
            ie.ie_linear_bwd_db(qt_to_dev(dY), db, ws)
            assert_same(db, o.linear_bwd_db(dY, group), f"db {group}")
    assert ws.status() == 0
