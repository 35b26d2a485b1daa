"""Calls of the block operators that share inputs (one tensor in two roles) or
run at once on two streams, each with a workspace of its own."""

import numpy as np
import pytest
import torch

import oracle as o
from integer_only_dnn_amd import ie
from tests.gpu_util import announce, assert_same, qt_to_dev, rand_qt

pytestmark = pytest.mark.gpu

EPS = o.Scalar(85, -23)
E = (EPS.mant, EPS.exp)


@pytest.mark.parametrize("shape", [(7, 96), (70, 200), (2100, 160)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("group", [o.TENSOR, o.ROW])
def test_one_tensor_in_two_roles(shape, group):
    announce(f"shared inputs {shape} {group}")
    M, N = shape
    rng = np.random.default_rng(M + N)
    ws = ie.Workspace("cuda")
    X, W, v = rand_qt(rng, (M, N), o.ROW), rand_qt(rng, (N, N), o.ROW), rand_qt(rng, (N, 1), o.ROW, -8, -4)
    Xd, Wd, vd = qt_to_dev(X), qt_to_dev(W), qt_to_dev(v)
    Y = ie.Mat.empty(M, N, group)
    ie.ie_linear_fwd_fused(Xd, Wd, vd, Xd, Y, ie.ACT_NONE, ws)
    assert_same(Y, o.linear_fwd_fused(X, W, v, X, group), "residual = input")
    if M <= 200:
        G = ie.Mat.empty(M, M, group)
        b = rand_qt(rng, (M, 1), o.TENSOR)
        ie.ie_linear_fwd_fused(Xd, Xd, qt_to_dev(b), None, G, ie.ACT_RELU, ws)
        assert_same(G, o.linear_fwd_fused(X, X, b, None, group, True), "weight = input")
    ie.ie_layer_norm_fwd(Xd, vd, vd, E, Y, ws)
    assert_same(Y, o.layer_norm_fwd(X, v, v, EPS, group), "gamma = beta")
    dg, db = ie.Mat.empty(N, 1, o.ROW), ie.Mat.empty(N, 1, o.ROW)
    ie.ie_layer_norm_bwd(Xd, Xd, vd, E, Y, dg, db, ws)
    for got, want, what in zip((Y, dg, db), o.layer_norm_bwd(X, X, v, EPS, group, o.ROW), ("dX", "dgamma", "dbeta")):
        assert_same(got, want, f"dY = X: {what}")
    ie.ie_dropout(Xd, Xd, Y, 9000, 5, 6, ws)
    assert_same(Y, o.dropout(X, X, 9000, 5, 6, group), "residual = input of dropout")
    assert ws.status() == 0


def test_two_streams_at_once():
    announce("two streams")
    rng = np.random.default_rng(4)
    sides = []
    for k, (M, N, K) in enumerate(((3000, 300, 96), (40, 500, 320))):
        X, W, b = rand_qt(rng, (M, K), o.ROW), rand_qt(rng, (N, K), o.ROW), rand_qt(rng, (N, 1), o.ROW)
        D = rand_qt(rng, (M, N), o.ROW, -10, 2)
        group = (o.ROW, o.TENSOR)[k]
        Y, Z, S, P = (ie.Mat.empty(M, N, group) for _ in range(4))
        dg, db, sb = (ie.Mat.empty(N, 1, group) for _ in range(3))
        sides.append(dict(host=(X, W, b, D, group), dev=[qt_to_dev(t) for t in (X, W, b, D)], out=(Y, Z, S, P, dg, db, sb),
                          ws=ie.Workspace("cuda"), stream=torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(6):
        for s in sides:
            X, W, b, D = s["dev"]
            Y, Z, S, P, dg, db, sb = s["out"]
            with torch.cuda.stream(s["stream"]):
                ie.ie_linear_fwd_fused(X, W, b, D, Y, ie.ACT_NONE, s["ws"])
                ie.ie_layer_norm_fwd(Y, b, b, E, Z, s["ws"])
                ie.ie_layer_norm_bwd(D, Y, b, E, S, dg, db, s["ws"])
                ie.ie_linear_bwd_db(D, sb, s["ws"])
                ie.ie_dropout(Z, Y, P, 20000, 3, i, s["ws"])
    torch.cuda.synchronize()
    for s in sides:
        X, W, b, D, g = s["host"]
        Y, Z, S, P, dg, db, sb = s["out"]
        y = o.linear_fwd_fused(X, W, b, D, g)
        z = o.layer_norm_fwd(y, b, b, EPS, g)
        dx, wg, wb = o.layer_norm_bwd(D, y, b, EPS, g, g)
        want = (y, z, dx, o.dropout(z, y, 20000, 3, 5, g), wg, wb, o.linear_bwd_db(D, g))
        for got, w, what in zip((Y, Z, S, P, dg, db, sb), want, ("product", "norm", "dX", "dropout", "dgamma", "dbeta", "db")):
            assert_same(got, w, what)
        with torch.cuda.stream(s["stream"]):
            assert s["ws"].status() == 0
