"""The transformer block's operators run together, as a training step uses
them: layer norm, product with bias and ReLU, product with bias, dropout onto
the residual stream; the backward pass through all of them; the update of
every parameter.  Three steps, every tensor against the oracle bit for bit,
eagerly and as a captured graph that draws anew on every replay."""

import numpy as np
import pytest
import torch

import oracle as o
from integer_only_dnn_amd import ie
from tests.gpu_util import announce, assert_same, qt_to_dev, rand_qt

pytestmark = pytest.mark.gpu

T, R = o.TENSOR, o.ROW
EPS, LR, MOM = (85, -23), (1, -7), (7, -3)
DROP, SEED = 6554, 0x1234567890ABCDEF


def inputs(rng, rows, dim, hidden):
    x = rand_qt(rng, (rows, dim), R, -8, -4)
    x.mant[rows - 1] = 0  # a padded token
    par = dict(gamma=rand_qt(rng, (dim, 1), R, -8, -7), beta=rand_qt(rng, (dim, 1), R, -9, -8),
               w1=rand_qt(rng, (hidden, dim), R, -11, -9), b1=rand_qt(rng, (hidden, 1), R, -9, -7),
               w2=rand_qt(rng, (dim, hidden), R, -12, -10), b2=rand_qt(rng, (dim, 1), R, -9, -7))
    vel = {k: o.QT(np.zeros_like(v.mant), np.full(v.mant.shape[0], o.E_MIN, np.int8), R) for k, v in par.items()}
    return x, rand_qt(rng, (rows, dim), R, -18, -14), par, vel


def oracle_step(x, dy, par, vel, step):
    eps = o.Scalar(*EPS)
    h = o.layer_norm_fwd(x, par["gamma"], par["beta"], eps, R)
    a = o.linear_fwd_fused(h, par["w1"], par["b1"], None, R, relu=True)
    z = o.linear_fwd_fused(a, par["w2"], par["b2"], None, R)
    y = o.dropout(z, x, DROP, SEED, step, R)
    dz = o.dropout(dy, None, DROP, SEED, step, R)
    g = dict(b2=o.linear_bwd_db(dz, R), w2=o.linear_bwd_dw(dz, a, R))
    da = o.linear_bwd_dx(dz, par["w2"], R)
    da = o.QT(o.relu_bwd(da.mant, a.mant).astype(np.int8), da.exp, R)
    g["b1"], g["w1"] = o.linear_bwd_db(da, R), o.linear_bwd_dw(da, h, R)
    dh = o.linear_bwd_dx(da, par["w1"], R)
    dn, g["gamma"], g["beta"] = o.layer_norm_bwd(dh, x, par["gamma"], eps, R, R)
    dx = o.sum_op(dn, dy, R)
    new = {k: o.sgd_update(par[k], vel[k], g[k], o.Scalar(*LR), o.Scalar(*MOM)) for k in par}
    return dict(h=h, a=a, z=z, y=y, dz=dz, da=da, dh=dh, dn=dn, dx=dx), g, {k: v[0] for k, v in new.items()}, \
        {k: v[1] for k, v in new.items()}


class Block:
    def __init__(self, x, dy, par, vel):
        rows, dim = x.mant.shape
        hidden = par["w1"].mant.shape[0]
        self.x, self.dy = qt_to_dev(x), qt_to_dev(dy)
        self.par = {k: qt_to_dev(v) for k, v in par.items()}
        self.vel = {k: qt_to_dev(v) for k, v in vel.items()}
        self.g = {k: ie.Mat.empty(*v.mant.shape, R) for k, v in par.items()}
        wide = ("a", "da")
        self.t = {k: ie.Mat.empty(rows, hidden if k in wide else dim, R)
                  for k in ("h", "a", "z", "y", "dz", "da", "dh", "dn", "dx")}
        self.ws = ie.Workspace("cuda")
        self.step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def run(self):
        p, t, g, ws = self.par, self.t, self.g, self.ws
        ie.ie_layer_norm_fwd(self.x, p["gamma"], p["beta"], EPS, t["h"], ws)
        ie.ie_linear_fwd_fused(t["h"], p["w1"], p["b1"], None, t["a"], ie.ACT_RELU, ws)
        ie.ie_linear_fwd_fused(t["a"], p["w2"], p["b2"], None, t["z"], ie.ACT_NONE, ws)
        ie.ie_dropout(t["z"], self.x, t["y"], DROP, SEED, 0, ws, self.step)
        ie.ie_dropout(self.dy, None, t["dz"], DROP, SEED, 0, ws, self.step)
        ie.ie_linear_bwd_db(t["dz"], g["b2"], ws)
        ie.ie_linear_bwd_dw(t["dz"], t["a"], g["w2"], ws)
        ie.ie_linear_bwd_dx_act(t["dz"], p["w2"], t["a"], t["da"], ie.ACT_RELU, ws)
        ie.ie_linear_bwd_db(t["da"], g["b1"], ws)
        ie.ie_linear_bwd_dw(t["da"], t["h"], g["w1"], ws)
        ie.ie_linear_bwd_dx(t["da"], p["w1"], t["dh"], ws)
        ie.ie_layer_norm_bwd(t["dh"], self.x, p["gamma"], EPS, t["dn"], g["gamma"], g["beta"], ws)
        ie.ie_add(t["dn"], self.dy, t["dx"], ws)
        names = sorted(p)
        ie.ie_sgd_update_multi([p[k] for k in names], [self.vel[k] for k in names], [g[k] for k in names], LR, MOM,
                               ws=ws)
        self.step += 1


def compare(block, want, g, par, vel, what):
    for k, v in want.items():
        assert_same(block.t[k], v, f"{what} {k}")
    for k in par:
        assert_same(block.g[k], g[k], f"{what} gradient of {k}")
        assert_same(block.par[k], par[k], f"{what} {k} updated")
        assert_same(block.vel[k], vel[k], f"{what} velocity of {k}")
    assert block.ws.status() == 0


@pytest.mark.parametrize("shape", [(50, 64, 160), (197, 192, 300), (33, 67, 129)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_block_trains(shape, graph):
    announce(f"block {shape} graph={graph}")
    rng = np.random.default_rng(sum(shape))
    x, dy, par, vel = inputs(rng, *shape)
    if graph:
        warm = Block(x, dy, par, vel)  # sizes the workspace on another block's state
        warm.run()
        torch.cuda.synchronize()
    block = Block(x, dy, par, vel)
    if graph:
        block.ws = warm.ws
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            block.run()
    for step in range(3):
        if graph:
            captured.replay()
        else:
            block.run()
        torch.cuda.synchronize()
        want, g, par, vel = oracle_step(x, dy, par, vel, step)
        compare(block, want, g, par, vel, f"step {step}")
