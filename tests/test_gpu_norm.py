"""GPU parity of layer norm (forward, backward, the sums of its parameters'
gradients) and of the bias gradient, bit for bit against the oracle: every
row length the kernels split differently, odd sizes, both groups of every
operand, flat, zero and padded rows, extreme exponents, unaligned buffers,
other streams and captured graphs."""

import numpy as np
import pytest
import torch

import oracle as o
from integer_only_dnn_amd import ie
from tests.gpu_util import announce, assert_same, qt_to_dev, rand_qt

pytestmark = pytest.mark.gpu

T, R = o.TENSOR, o.ROW
EPS = o.Scalar(85, -23)
SHAPES = [(1, 1), (1, 2), (3, 5), (7, 64), (33, 65), (64, 256), (129, 257), (50, 385), (50, 512), (31, 513),
          (40, 768), (9, 1023), (9, 1025), (5, 2049), (5, 4096), (4, 4097), (3, 8195), (2, 12289), (2, 16384),
          (3000, 192), (2100, 30), (0, 8), (4, 0)]


@pytest.fixture(scope="module")
def ws():
    return ie.Workspace("cuda")


def vec(rng, n, kind):
    if kind is None:
        return None
    if kind == "1":
        return o.QT(rng.integers(-128, 128, (1, n)).astype(np.int8), np.array([-7], np.int8), R)
    return rand_qt(rng, (n, 1), kind, -10, -5)


def dev(v):
    return None if v is None else qt_to_dev(v)


def check(X, dY, gam, bet, groups, vg, ws, eps=EPS, bits=8, what=""):
    """Forward and backward of one input; groups: of Y and dX, vg: of the gradients of the parameters."""
    rows, cols = X.mant.shape
    e = (eps.mant, eps.exp)
    Xd, dYd, gd, bd = qt_to_dev(X), qt_to_dev(dY), dev(gam), dev(bet)
    Y = ie.Mat.empty(rows, cols, groups[0], bits=bits)
    ie.ie_layer_norm_fwd(Xd, gd, bd, e, Y, ws)
    assert_same(Y, o.layer_norm_fwd(X, gam, bet, eps, groups[0], bits), what + " Y")
    dX = ie.Mat.empty(rows, cols, groups[1], bits=bits)
    dg, db = ie.Mat.empty(cols, 1, vg, bits=bits), ie.Mat.empty(cols, 1, vg, bits=bits)
    ie.ie_layer_norm_bwd(dYd, Xd, gd, e, dX, dg, db, ws)
    want = o.layer_norm_bwd(dY, X, gam, eps, groups[1], vg, bits)
    for m, w, name in zip((dX, dg, db), want, ("dX", "dgamma", "dbeta")):
        assert_same(m, w, what + " " + name)
    assert ws.status() == 0


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("groups", [(T, T, T, T, T), (R, R, R, R, R), (R, T, T, R, T)], ids=["T", "R", "RTTRT"])
def test_norm_shapes(shape, groups, ws):
    announce(f"norm {shape} {groups}")
    rng = np.random.default_rng(shape[0] * 7 + shape[1])
    X, dY = rand_qt(rng, shape, groups[0]), rand_qt(rng, shape, groups[1], -20, -9)
    kind = R if groups[4] == R else T
    gam, bet = vec(rng, shape[1], kind), vec(rng, shape[1], kind)
    if shape[1] == 0:  # no channels: only the exponents are there
        gam = bet = None
        rows = shape[0]
        Y, dX = ie.Mat.empty(rows, 0, groups[2]), ie.Mat.empty(rows, 0, groups[3])
        ie.ie_layer_norm_fwd(qt_to_dev(X, rows=rows), None, None, (1, -20), Y, ws)
        ie.ie_layer_norm_bwd(qt_to_dev(dY, rows=rows), qt_to_dev(X, rows=rows), None, (1, -20), dX, None, None, ws)
        torch.cuda.synchronize()
        assert bool((Y.exp == o.E_MIN).all()) and bool((dX.exp == o.E_MIN).all())
        return
    check(X, dY, gam, bet, groups[2:4], groups[4], ws, what=str(shape))


@pytest.mark.parametrize("kind", [None, T, R, "1"], ids=["none", "T", "R", "1xN"])
@pytest.mark.parametrize("bits", [8, 4, 2])
def test_norm_parameters_and_widths(kind, bits, ws):
    announce(f"norm parameters {kind} bits {bits}")
    rng = np.random.default_rng(bits)
    X, dY = rand_qt(rng, (37, 100), R), rand_qt(rng, (37, 100), R, -20, -9)
    check(X, dY, vec(rng, 100, kind), vec(rng, 100, kind), (R, T), R if bits == 8 else T, ws, bits=bits)


def test_norm_outputs_can_be_skipped(ws):
    announce("norm backward, outputs skipped")
    rng = np.random.default_rng(1)
    X, dY, gam = rand_qt(rng, (70, 40), R), rand_qt(rng, (70, 40), R), vec(rng, 40, R)
    want = o.layer_norm_bwd(dY, X, gam, EPS, T, R)
    e = (EPS.mant, EPS.exp)
    for mask in range(8):
        outs = [ie.Mat.empty(70, 40, T), ie.Mat.empty(40, 1, R), ie.Mat.empty(40, 1, R)]
        outs = [m if mask >> i & 1 else None for i, m in enumerate(outs)]
        ie.ie_layer_norm_bwd(qt_to_dev(dY), qt_to_dev(X), dev(gam), e, *outs, ws)
        for m, w in zip(outs, want):
            if m is not None:
                assert_same(m, w, f"mask {mask}")


@pytest.mark.parametrize("eps", [o.Scalar(0, 0), o.Scalar(1, -100), o.Scalar(127, 127), o.Scalar(85, -23)],
                         ids=["0", "2^-100", "huge", "1e-5"])
def test_norm_flat_and_extreme_rows(eps, ws):
    """Rows of one value, of zeros, of -128, with one odd element; exponents
    at both ends, so that eps is nothing, everything or in between."""
    announce(f"norm flat and extreme rows eps {eps}")
    rng = np.random.default_rng(2)
    n = 48
    rows = [np.full(n, 5), np.zeros(n), np.full(n, -128), np.r_[np.full(n - 1, 127), 126], np.r_[1, np.zeros(n - 1)],
            np.where(np.arange(n) % 2, 127, -128), rng.integers(-128, 128, n), rng.integers(-1, 2, n)]
    m = np.array(rows).astype(np.int8)
    for ex in (-128, -60, 0, 60, 127):
        X = o.QT(m, np.full(len(rows), ex, np.int8), R)
        dY = rand_qt(rng, m.shape, R, -20, -9)
        dY.mant[5] = 0
        gam, bet = vec(rng, n, R), vec(rng, n, T)
        Y = ie.Mat.empty(*m.shape, R)
        ie.ie_layer_norm_fwd(qt_to_dev(X), dev(gam), dev(bet), (eps.mant, eps.exp), Y, ws)
        assert_same(Y, o.layer_norm_fwd(X, gam, bet, eps, R), f"Y e={ex}")
        dX, dg, db = ie.Mat.empty(*m.shape, R), ie.Mat.empty(n, 1, R), ie.Mat.empty(n, 1, T)
        try:
            want = o.layer_norm_bwd(dY, X, gam, eps, R, R)
        except o.ExpRangeError:
            ie.ie_layer_norm_bwd(qt_to_dev(dY), qt_to_dev(X), dev(gam), (eps.mant, eps.exp), dX, dg, db, ws)
            assert ws.status() == ie.FLAG_EXP_RANGE
            continue
        ie.ie_layer_norm_bwd(qt_to_dev(dY), qt_to_dev(X), dev(gam), (eps.mant, eps.exp), dX, dg, db, ws)
        assert_same(dX, want[0], f"dX e={ex}")
        assert_same(dg, want[1], f"dgamma e={ex}")
        assert ws.status() == 0


def test_norm_exponent_range_is_flagged(ws):
    announce("norm exponent range")
    X = o.QT(np.array([[127, -127]], np.int8), np.array([0], np.int8), R)
    gam = o.QT(np.array([[127], [127]], np.int8), np.array([127], np.int8), T)
    for group in (R, T):
        Y = ie.Mat.empty(1, 2, group)
        ie.ie_layer_norm_fwd(qt_to_dev(X), dev(gam), dev(gam), (1, -20), Y, ws)
        assert ws.status() == ie.FLAG_EXP_RANGE and ws.status() == 0


def _shifted(t, k):
    """The same data at an address k bytes past a 16-byte boundary, exponents too."""
    def at(a):
        buf = torch.empty(a.size + 16, dtype=torch.int8, device="cuda")
        v = buf[k:k + a.size].view(a.shape)
        v.copy_(torch.from_numpy(a))
        return v
    return ie.Mat(at(np.ascontiguousarray(t.mant)), at(np.ascontiguousarray(t.exp)), t.group)


@pytest.mark.parametrize("shape", [(19, 64), (19, 67), (3, 4099)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("k", [1, 2, 3])
def test_norm_unaligned_buffers(shape, k, ws):
    announce(f"norm {shape} buffers off by {k}")
    rng = np.random.default_rng(k)
    X, dY = rand_qt(rng, shape, R), rand_qt(rng, shape, R)
    gam, bet = vec(rng, shape[1], R), vec(rng, shape[1], R)
    e = (EPS.mant, EPS.exp)
    zero = o.QT(np.zeros(shape, np.int8), np.zeros(shape[0], np.int8), R)
    zv = o.QT(np.zeros((shape[1], 1), np.int8), np.zeros(shape[1], np.int8), R)
    Y, dX, dg, db = _shifted(zero, k), _shifted(zero, k), _shifted(zv, k), _shifted(zv, k)
    Xd, dYd, gd, bd = (_shifted(t, k) for t in (X, dY, gam, bet))
    ie.ie_layer_norm_fwd(Xd, gd, bd, e, Y, ws)
    ie.ie_layer_norm_bwd(dYd, Xd, gd, e, dX, dg, db, ws)
    assert_same(Y, o.layer_norm_fwd(X, gam, bet, EPS, R), "Y")
    for m, w, name in zip((dX, dg, db), o.layer_norm_bwd(dY, X, gam, EPS, R, R), ("dX", "dgamma", "dbeta")):
        assert_same(m, w, name)
    ie.ie_linear_bwd_db(dYd, db, ws)
    assert_same(db, o.linear_bwd_db(dY, R), "db")


@pytest.mark.parametrize("shape", [(1, 1), (3, 5), (64, 256), (129, 257), (2000, 30), (33, 1000), (5, 20000), (0, 8),
                                   (4, 0), (40000, 3)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("groups", [(T, T), (R, R), (R, T)], ids=["TT", "RR", "RT"])
def test_bias_gradient(shape, groups, ws):
    announce(f"db {shape} {groups}")
    rng = np.random.default_rng(shape[0] + shape[1])
    dY = rand_qt(rng, shape, groups[0], -40, -9)
    db = ie.Mat.empty(shape[1], 1, groups[1])
    ie.ie_linear_bwd_db(qt_to_dev(dY) if shape[1] else qt_to_dev(dY, rows=shape[0]), db, ws)
    if shape[1] == 0:
        torch.cuda.synchronize()
        assert bool((db.exp == o.E_MIN).all())
        return
    assert_same(db, o.linear_bwd_db(dY, groups[1]), str(shape))
    one = ie.Mat.empty(1, shape[1], R)
    ie.ie_linear_bwd_db(qt_to_dev(dY), one, ws)
    want = o.linear_bwd_db(dY, T)
    assert_same(one, o.QT(want.mant.reshape(1, -1), want.exp, R), "1xN")


def test_norm_far_exponents(ws):
    """Rows of dY 40 and more exponents apart: the small ones vanish from the
    column sums but not from dX; the same with gamma's channels."""
    announce("norm far exponents")
    rng = np.random.default_rng(4)
    X, dY = rand_qt(rng, (8, 20), R), rand_qt(rng, (8, 20), R)
    dY = o.QT(dY.mant, np.array([-128, -100, -40, -10, -9, 0, 30, 31], np.int8), R)
    gam = o.QT(rng.integers(-128, 128, (20, 1)).astype(np.int8), rng.integers(-128, 10, 20).astype(np.int8), R)
    check(X, dY, gam, gam, (R, R), R, ws)


def test_norm_other_stream_and_graph(ws):
    """On a stream of its own, and captured: every replay on new inputs."""
    announce("norm stream and graph")
    rng = np.random.default_rng(6)
    shape, e = (300, 200), (EPS.mant, EPS.exp)
    gam, bet = vec(rng, 200, R), vec(rng, 200, R)
    gd, bd = dev(gam), dev(bet)
    Xd, dYd = qt_to_dev(rand_qt(rng, shape, R)), qt_to_dev(rand_qt(rng, shape, R))
    Y, dX = ie.Mat.empty(*shape, T), ie.Mat.empty(*shape, T)
    dg, db, dl = (ie.Mat.empty(200, 1, T) for _ in range(3))
    own = ie.Workspace("cuda")

    def step():
        ie.ie_layer_norm_fwd(Xd, gd, bd, e, Y, own)
        ie.ie_layer_norm_bwd(dYd, Xd, gd, e, dX, dg, db, own)
        ie.ie_linear_bwd_db(dYd, dl, own)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        X, dY = rand_qt(rng, shape, R), rand_qt(rng, shape, R, -30, -9)
        for d, h in ((Xd, X), (dYd, dY)):
            d.mant.copy_(torch.from_numpy(h.mant))
            d.exp.copy_(torch.from_numpy(h.exp))
        graph.replay()
        torch.cuda.synchronize()
        assert_same(Y, o.layer_norm_fwd(X, gam, bet, EPS, T), "replayed Y")
        for m, w, name in zip((dX, dg, db), o.layer_norm_bwd(dY, X, gam, EPS, T, T), ("dX", "dgamma", "dbeta")):
            assert_same(m, w, "replayed " + name)
        assert_same(dl, o.linear_bwd_db(dY, T), "replayed db")
    assert own.status() == 0


def test_norm_leaves_what_is_not_its_own(ws):
    """Bytes before and behind every output stay as they were."""
    announce("norm guard bytes")
    rng = np.random.default_rng(8)
    e = (EPS.mant, EPS.exp)
    for shape in ((5, 67), (17, 192), (3, 1026)):
        X, dY = rand_qt(rng, shape, R), rand_qt(rng, shape, R)
        gam = vec(rng, shape[1], R)
        bufs, mats = [], []
        for r, c in (shape, shape, (shape[1], 1), (shape[1], 1)):
            pair = [torch.full((n + 128,), 77, dtype=torch.int8, device="cuda") for n in (r * c, r)]
            bufs += pair
            mats.append(ie.Mat(pair[0][64:64 + r * c].view(r, c), pair[1][64:64 + r], R))
        Y, dX, dg, db = mats
        ie.ie_layer_norm_fwd(qt_to_dev(X), dev(gam), None, e, Y, ws)
        ie.ie_layer_norm_bwd(qt_to_dev(dY), qt_to_dev(X), dev(gam), e, dX, dg, db, ws)
        torch.cuda.synchronize()
        for b in bufs:
            assert bool((b[:64] == 77).all()) and bool((b[-64:] == 77).all())
        assert_same(dX, o.layer_norm_bwd(dY, X, gam, EPS, R, R)[0], "dX")


# whole-tensor results that one block holds, and one past each edge of that;
# few partial rows of column sums; one row
ONE = [(1, 1), (1, 300), (1, 5000), (16, 1024), (17, 1000), (16, 1025), (64, 256), (65, 250), (64, 257), (50, 61),
       (40, 130), (8, 777), (9, 900), (33, 192), (128, 1000), (129, 4096), (100, 4097)]


@pytest.mark.parametrize("shape", ONE, ids=lambda s: "x".join(map(str, s)))
def test_norm_small_whole_tensor_results(shape, ws):
    M, N = shape
    announce(f"norm one block {shape}")
    rng = np.random.default_rng(M * 7 + N)
    for xg, vg in ((o.ROW, o.ROW), (o.TENSOR, o.TENSOR)):
        X, dY = rand_qt(rng, (M, N), xg), rand_qt(rng, (M, N), xg, -20, 3)
        X.mant[M // 2], dY.mant[M // 3] = 5, 0
        g, b = rand_qt(rng, (N, 1), vg, -8, -4), rand_qt(rng, (N, 1), vg, -8, -4)
        e = (EPS.mant, EPS.exp)
        Y = ie.Mat.empty(M, N, o.TENSOR)
        ie.ie_layer_norm_fwd(qt_to_dev(X), qt_to_dev(g), qt_to_dev(b), e, Y, ws)
        assert_same(Y, o.layer_norm_fwd(X, g, b, EPS, o.TENSOR), f"fwd {shape}")
        dX, dg, db = ie.Mat.empty(M, N, o.TENSOR), ie.Mat.empty(N, 1, vg), ie.Mat.empty(N, 1, o.TENSOR)
        ie.ie_layer_norm_bwd(qt_to_dev(dY), qt_to_dev(X), qt_to_dev(g), e, dX, dg, db, ws)
        want = o.layer_norm_bwd(dY, X, g, EPS, o.TENSOR, vg)[:2] + o.layer_norm_bwd(dY, X, g, EPS, o.TENSOR, o.TENSOR)[2:]
        for got, w, what in zip((dX, dg, db), want, "xgb"):
            assert_same(got, w, f"bwd {shape} {what}")
        s = ie.Mat.empty(N, 1, o.TENSOR)
        ie.ie_linear_bwd_db(qt_to_dev(dY), s, ws)
        assert_same(s, o.linear_bwd_db(dY, o.TENSOR), f"sums {shape}")
    assert ws.status() == 0


@pytest.mark.parametrize("shape", [(65536, 3), (70001, 7), (131073, 16)], ids=lambda s: "x".join(map(str, s)))
def test_norm_many_rows(shape, ws):
    """The rows' largest exponent found by a launch of its own, and one row short of that."""
    announce(f"norm many rows {shape}")
    M, N = shape
    rng = np.random.default_rng(M)
    X, dY = rand_qt(rng, (M, N), o.ROW), rand_qt(rng, (M, N), o.ROW, -20, -9)
    dY.exp[M - 1] = -5  # the largest, in the last row
    check(X, dY, None, None, (o.ROW, o.TENSOR), o.ROW, ws, what=str(shape))
    s = ie.Mat.empty(N, 1, o.ROW)
    ie.ie_linear_bwd_db(qt_to_dev(dY), s, ws)
    assert_same(s, o.linear_bwd_db(dY, o.ROW), str(shape))
