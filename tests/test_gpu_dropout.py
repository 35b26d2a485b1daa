"""GPU parity of dropout bit for bit against the oracle: every row length the
kernels split differently, odd and unaligned rows, all groups, with and
without the residual, rates at both ends, the gradient's mask, steps read
from device memory, other streams and captured graphs."""

import ctypes

import numpy as np
import pytest
import torch

import oracle as o
from integer_only_dnn_amd import ie
from tests.gpu_util import announce, assert_same, qt_to_dev, rand_qt

pytestmark = pytest.mark.gpu

T, R = o.TENSOR, o.ROW
SEED = 0xFEDCBA9876543210
SHAPES = [(1, 1), (5, 7), (33, 8), (40, 65), (64, 128), (21, 193), (30, 257), (19, 385), (9, 513), (10, 768),
          (5, 1025), (3, 1537), (3, 2049), (2, 4097), (2, 6145), (2, 8193), (1, 16385), (2, 24576), (2, 24577),
          (3000, 3), (0, 5), (4, 0)]


@pytest.fixture(scope="module")
def ws():
    return ie.Workspace("cuda")


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("groups", [(T, None, T), (R, None, R), (R, T, R), (T, R, T), (R, R, T)],
                         ids=["T-T", "R-R", "RTR", "TRT", "RRT"])
def test_dropout_shapes(shape, groups, ws):
    announce(f"dropout {shape} {groups}")
    rng = np.random.default_rng(shape[0] + 3 * shape[1])
    rows, cols = shape
    X = rand_qt(rng, shape, groups[0])
    D = None if groups[1] is None else rand_qt(rng, shape, groups[1])
    Y = ie.Mat.empty(rows, cols, groups[2])
    to = lambda t: None if t is None else qt_to_dev(t, rows=rows) if cols == 0 else qt_to_dev(t)  # noqa: E731
    ie.ie_dropout(to(X), to(D), Y, 13107, SEED, 5, ws)
    if cols == 0:
        torch.cuda.synchronize()
        assert bool((Y.exp == o.E_MIN).all())
        return
    assert_same(Y, o.dropout(X, D, 13107, SEED, 5, groups[2]), str(shape))
    assert ws.status() == 0


@pytest.mark.parametrize("drop", [0, 1, 32768, 60000, 65535])
@pytest.mark.parametrize("bits", [8, 3])
def test_dropout_rates_seeds_and_steps(drop, bits, ws):
    announce(f"dropout drop {drop} bits {bits}")
    rng = np.random.default_rng(drop)
    X, D = rand_qt(rng, (20, 50), R), rand_qt(rng, (20, 50), R)
    for seed, step in ((0, 0), ((1 << 64) - 1, (1 << 64) - 1), (1 << 32, 1), (1, 1 << 32)):
        Y, Z = ie.Mat.empty(20, 50, R, bits=bits), ie.Mat.empty(20, 50, T, bits=bits)
        ie.ie_dropout(qt_to_dev(X), qt_to_dev(D), Y, drop, seed, step, ws)
        ie.ie_dropout(qt_to_dev(X), None, Z, drop, seed, step, ws)
        assert_same(Y, o.dropout(X, D, drop, seed, step, R, bits), "with residual")
        assert_same(Z, o.dropout(X, None, drop, seed, step, T, bits), "alone")


def test_dropout_far_exponents(ws):
    """The residual far above, far below and next to the input; zero and
    dropped-out rows; the ends of the exponent range."""
    announce("dropout far exponents")
    rng = np.random.default_rng(3)
    e = np.array([-128, -128, -60, -40, -20, 0, 20, 60, 120, 126], np.int8)
    X = o.QT(rng.integers(-128, 128, (10, 24)).astype(np.int8), e, R)
    X.mant[4] = 0
    for re in (-128, -60, -3, 0, 60, 120):
        D = o.QT(rng.integers(-128, 128, (10, 24)).astype(np.int8), np.full(10, re, np.int8), R)
        D.mant[5] = 0
        Y = ie.Mat.empty(10, 24, R)
        ie.ie_dropout(qt_to_dev(X), qt_to_dev(D), Y, 30000, 7, 9, ws)
        try:
            want = o.dropout(X, D, 30000, 7, 9, R)
        except o.ExpRangeError:
            assert ws.status() == ie.FLAG_EXP_RANGE
            continue
        assert_same(Y, want, f"residual at {re}")
        assert ws.status() == 0


def test_dropout_backward_is_the_same_mask(ws):
    """The gradient keeps what the forward pass kept, scaled alike."""
    announce("dropout backward")
    rng = np.random.default_rng(4)
    ones = o.QT(np.full((60, 70), 64, np.int8), np.array([-6], np.int8), T)
    dY = rand_qt(rng, (60, 70), R)
    Y, dX = ie.Mat.empty(60, 70, T), ie.Mat.empty(60, 70, R)
    ie.ie_dropout(qt_to_dev(ones), None, Y, 32768, SEED, 11, ws)
    ie.ie_dropout(qt_to_dev(dY), None, dX, 32768, SEED, 11, ws)
    torch.cuda.synchronize()
    keep = Y.mant.cpu().numpy() != 0
    assert 0.4 < keep.mean() < 0.6
    got = np.ldexp(dX.mant.cpu().numpy().astype(float), dX.exp.cpu().numpy()[:, None].astype(int))
    want = np.where(keep, 2 * np.ldexp(dY.mant.astype(float), dY.exp[:, None].astype(int)), 0)
    # doubling is exact, but a row that keeps a -128 takes the next exponent (|C| <= 127: 128 rounds to 64 there), so
    # each result is off by at most half a unit of its row's exponent; what is dropped is exactly 0
    unit = np.ldexp(1.0, dX.exp.cpu().numpy()[:, None].astype(int))
    off = np.abs(got - want)
    assert (off <= unit / 2).all() and not got[~keep].any()
    rows = (np.where(keep, dY.mant, 0) == -128).any(axis=1)
    assert not off[~rows].any()


@pytest.mark.parametrize("k", [1, 2, 3])
def test_dropout_unaligned_buffers_and_guards(k, ws):
    announce(f"dropout buffers off by {k}")
    rng = np.random.default_rng(k)
    for shape in ((7, 61), (4, 64), (2, 24579)):
        X, D = rand_qt(rng, shape, R), rand_qt(rng, shape, R)

        def at(a, fill=False):
            buf = torch.full((a.size + 64,), 77, dtype=torch.int8, device="cuda")
            v = buf[16 + k:16 + k + a.size].view(a.shape)
            if not fill:
                v.copy_(torch.from_numpy(a))
            return buf, v
        mk = lambda t: ie.Mat(at(t.mant)[1], at(t.exp)[1], t.group)  # noqa: E731
        (bm, vm), (be, ve) = at(X.mant, True), at(X.exp, True)
        Y = ie.Mat(vm, ve, R)
        ie.ie_dropout(mk(X), mk(D), Y, 6554, 1, 2, ws)
        assert_same(Y, o.dropout(X, D, 6554, 1, 2, R), str(shape))
        for b, n in ((bm, X.mant.size), (be, X.exp.size)):
            assert bool((b[:16 + k] == 77).all()) and bool((b[16 + k + n:] == 77).all())


def test_dropout_stream_and_graph_with_a_device_step():
    """Captured once; the step in device memory moves on between replays."""
    announce("dropout stream and graph")
    rng = np.random.default_rng(6)
    X, D = rand_qt(rng, (90, 100), R), rand_qt(rng, (90, 100), T)
    Xd, Dd, Y, Z = qt_to_dev(X), qt_to_dev(D), ie.Mat.empty(90, 100, R), ie.Mat.empty(90, 100, T)
    own, step = ie.Workspace("cuda"), torch.tensor([3], dtype=torch.int64, device="cuda")

    def run():
        ie.ie_dropout(Xd, Dd, Y, 6554, SEED, 1 << 40, own, step)
        ie.ie_dropout(Xd, None, Z, 6554, SEED, 1, own, step)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        run()
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(4):
        step.fill_(3 + 5 * i)
        graph.replay()
        torch.cuda.synchronize()
        assert_same(Y, o.dropout(X, D, 6554, SEED, (1 << 40) + 3 + 5 * i, R), f"replay {i}")
        assert_same(Z, o.dropout(X, None, 6554, SEED, 4 + 5 * i, T), f"replay {i}")


def test_dropout_refusals_on_the_binding(ws):
    X, Y = qt_to_dev(rand_qt(np.random.default_rng(0), (4, 8), T)), ie.Mat.empty(4, 8, T)
    for bad in (dict(drop=-1), dict(seed=-1), dict(step=1 << 64), dict(step_ptr=torch.zeros(1, dtype=torch.int64))):
        with pytest.raises(ValueError):
            ie.ie_dropout(X, None, Y, **{**dict(drop=1, seed=1, step=1, ws=ws), **bad})
    with pytest.raises(ie.IeError):
        ie.ie_dropout(X, None, Y, 65536, 1, 1, ws)
    assert ctypes.sizeof(ie.ie_dropout_desc) == 32
