"""GPU parity of the product with bias, residual and ReLU bit for bit against
the oracle: every plan (direct, round to odd, split), odd sizes, all groups,
bias and residual present or absent, exponents next to and far from the
product's, unaligned buffers, single rows, empty contractions, other streams
and captured graphs."""

import itertools

import numpy as np
import pytest
import torch

import oracle as o
from integer_only_dnn_amd import ie
from tests.gpu_util import announce, assert_same, qt_to_dev, rand_qt

pytestmark = pytest.mark.gpu

T, R = o.TENSOR, o.ROW


@pytest.fixture(scope="module")
def ws():
    return ie.Workspace("cuda")


def vec(rng, n, kind, elo=-12, ehi=-5):
    return None if kind is None else rand_qt(rng, (n, 1), kind, elo, ehi)


def dev(t):
    return None if t is None else qt_to_dev(t)


def check(X, W, b, D, yg, relu, ws, bits=8, what=""):
    M, N = X.mant.shape[0], W.mant.shape[0]
    Y = ie.Mat.empty(M, N, yg, bits=bits)
    ie.ie_linear_fwd_fused(qt_to_dev(X), qt_to_dev(W), dev(b), dev(D), Y, ie.ACT_RELU if relu else ie.ACT_NONE, ws)
    assert_same(Y, o.linear_fwd_fused(X, W, b, D, yg, relu, bits), what)
    assert ws.status() == 0


# (M, N, K): one tile, tile edges, rows of one 64 x 256 tile, rows over several
# tiles, split contractions, single tokens, K below and off the padding
SHAPES = [(1, 1, 1), (3, 5, 7), (64, 64, 128), (64, 128, 256), (65, 129, 130), (200, 200, 96), (130, 256, 64),
          (513, 257, 160), (1, 4096, 1024), (5, 1000, 2048), (7, 33, 4096), (40, 300, 1040), (260, 31, 16),
          (1300, 700, 48), (4000, 130, 272)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("groups", [(T, T, T, T, T), (R, R, R, R, R), (R, T, R, T, T), (T, R, T, R, R)],
                         ids=["T", "R", "RTRTT", "TRTRR"])
def test_linear_fused_shapes(shape, groups, ws):
    M, N, K = shape
    announce(f"linear fused {shape} {groups}")
    rng = np.random.default_rng(M + N + K)
    X, W = rand_qt(rng, (M, K), groups[0]), rand_qt(rng, (N, K), groups[1])
    b, D = vec(rng, N, groups[2]), rand_qt(rng, (M, N), groups[3], -10, 2)
    for relu, bb, dd in ((True, b, D), (False, b, None), (False, None, D)):
        check(X, W, bb, dd, groups[4], relu, ws, what=f"{shape} relu={relu}")


def test_linear_fused_without_addends_is_the_plain_product(ws):
    announce("linear fused, plain")
    rng = np.random.default_rng(1)
    for (M, N, K), yg in itertools.product([(70, 300, 96), (5, 64, 2048)], (T, R)):
        X, W = rand_qt(rng, (M, K), R), rand_qt(rng, (N, K), R)
        for act in (ie.ACT_NONE, ie.ACT_RELU):
            Y, Z = ie.Mat.empty(M, N, yg), ie.Mat.empty(M, N, yg)
            ie.ie_linear_fwd_fused(qt_to_dev(X), qt_to_dev(W), None, None, Y, act, ws)
            ie.ie_linear_fwd_act(qt_to_dev(X), qt_to_dev(W), Z, act, ws)
            torch.cuda.synchronize()
            assert torch.equal(Y.mant, Z.mant) and torch.equal(Y.exp, Z.exp)


@pytest.mark.parametrize("plan", ["2,2,1", "1,4,1", "2,1,1", "1,1,1", "1,1,2,3", "2,2,2,2", "2,2,0", "1,4,0", "2,1,0",
                                  "1,1,0"])
@pytest.mark.parametrize("yg", [T, R])
def test_linear_fused_plans(plan, yg, ws, monkeypatch):
    """Every built plan on one shape; direct ones where a group fits a tile."""
    announce(f"linear fused plan {plan} group {yg}")
    rng = np.random.default_rng(2)
    direct = plan.endswith(",0")
    M, N, K = (50, 60, 300) if direct else (140, 300, 520)
    X, W = rand_qt(rng, (M, K), R), rand_qt(rng, (N, K), R)
    b, D = vec(rng, N, R), rand_qt(rng, (M, N), R, -10, 2)
    monkeypatch.setenv("IE_TILE", plan)
    for relu, bb, dd in ((True, b, D), (False, b, None), (False, None, D)):
        check(X, W, bb, dd, yg, relu, ws, what=plan)


def test_linear_fused_refuses_plans_that_are_not_built(ws, monkeypatch):
    rng = np.random.default_rng(2)
    X, W, b = rand_qt(rng, (140, 64), R), rand_qt(rng, (300, 64), R), vec(rng, 300, R)
    for plan in ("2,2,3", "4,1,1", "2,2,0"):
        monkeypatch.setenv("IE_TILE", plan)
        with pytest.raises(ie.IeError):
            ie.ie_linear_fwd_fused(qt_to_dev(X), qt_to_dev(W), qt_to_dev(b), None, ie.Mat.empty(140, 300, R), 0, ws)


@pytest.mark.parametrize("bits", [7, 4, 2])
@pytest.mark.parametrize("shape", [(66, 130, 64), (6, 70, 2048)], ids=["rto", "split"])
def test_linear_fused_widths(bits, shape, ws):
    announce(f"linear fused bits {bits} {shape}")
    M, N, K = shape
    rng = np.random.default_rng(bits)
    X, W = rand_qt(rng, (M, K), R), rand_qt(rng, (N, K), T)
    b, D = vec(rng, N, R), rand_qt(rng, (M, N), T, -8, -2)
    for yg in (T, R):
        check(X, W, b, D, yg, True, ws, bits=bits)


@pytest.mark.parametrize("gap", [-120, -60, -40, -25, -8, 0, 8, 25, 40, 60, 120])
@pytest.mark.parametrize("shape", [(66, 140, 64), (6, 70, 2048), (50, 200, 64)], ids=["rto", "split", "direct"])
def test_linear_fused_far_exponents(gap, shape, ws):
    """Bias and residual far above and far below the product, and far from
    each other; rows and columns of zeros; -128 everywhere."""
    announce(f"linear fused gap {gap} {shape}")
    M, N, K = shape
    rng = np.random.default_rng(gap + 200)
    X, W = rand_qt(rng, (M, K), R, -6, -6), rand_qt(rng, (N, K), R, -6, -6)
    X.mant[1], W.mant[2], X.mant[3], W.mant[3] = 0, 0, -128, -128
    e = np.clip(-12 + gap, -128, 110)
    b = o.QT(rng.integers(-128, 128, (N, 1)).astype(np.int8), np.full(N, e, np.int8), R)
    b.mant[::3] = 0
    D = o.QT(rng.integers(-128, 128, (M, N)).astype(np.int8), np.full(M, np.clip(-12 - gap, -128, 110), np.int8), R)
    D.mant[1], D.mant[:, 5] = 0, 0
    for yg, bb, dd in ((R, b, D), (T, b, D), (R, b, None), (R, None, D)):
        check(X, W, bb, dd, yg, False, ws, what=f"gap {gap}")


def test_linear_fused_ties_decided_by_the_bias(ws):
    """Sums that fall on a rounding tie, or a hair beside one."""
    announce("linear fused ties")
    # acc = 2 c + 1 at 2^-1 of the result's unit: a tie; the bias adds -1, 0 or 1 unit 30 places below
    n = 96
    X = o.QT(np.ones((1, 1), np.int8), np.array([0], np.int8), T)
    w = np.zeros((n, 1), np.int8)
    w[:, 0] = 2 * np.arange(n) % 126 + 1
    w[0, 0] = 127
    W = o.QT(w, np.array([0], np.int8), T)
    b = o.QT((np.arange(n) % 3 - 1).astype(np.int8).reshape(-1, 1), np.array([-30], np.int8), T)
    D = o.QT(np.zeros((1, n), np.int8), np.array([0], np.int8), T)
    D.mant[0, 0] = 127  # the group's largest: 254, so the unit is 2
    for yg in (T, R):
        check(X, W, b, D, yg, False, ws)


def test_linear_fused_empty_and_single(ws):
    announce("linear fused empty")
    rng = np.random.default_rng(3)
    b, D = vec(rng, 6, R), rand_qt(rng, (4, 6), R)
    X0, W0 = o.QT(np.zeros((4, 0), np.int8), np.zeros(4, np.int8), R), o.QT(np.zeros((6, 0), np.int8), np.zeros(6, np.int8), R)
    Y = ie.Mat.empty(4, 6, R)
    ie.ie_linear_fwd_fused(qt_to_dev(X0, rows=4), qt_to_dev(W0, rows=6), dev(b), dev(D), Y, 0, ws)
    assert_same(Y, o.linear_fwd_fused(X0, W0, b, D, R), "K = 0")
    E = ie.Mat.empty(0, 6, T)
    ie.ie_linear_fwd_fused(ie.Mat.empty(0, 16, R), dev(rand_qt(rng, (6, 16), R)), dev(b), None, E, 0, ws)
    torch.cuda.synchronize()
    assert int(E.exp[0]) == o.E_MIN


@pytest.mark.parametrize("k", [1, 2, 3, 8])
@pytest.mark.parametrize("shape", [(70, 61, 64), (70, 64, 64), (66, 323, 32), (5, 63, 2048)],
                         ids=lambda s: "x".join(map(str, s)))
def test_linear_fused_unaligned_and_guards(k, shape, ws):
    """Residual, bias and result at odd addresses; nothing written beside the result."""
    announce(f"linear fused {shape} off by {k}")
    M, N, K = shape
    rng = np.random.default_rng(k)
    X, W = rand_qt(rng, (M, K), R), rand_qt(rng, (N, K), R)
    b, D = vec(rng, N, R), rand_qt(rng, (M, N), R, -10, 2)

    def at(a, fill=False):
        buf = torch.full((a.size + 64,), 77, dtype=torch.int8, device="cuda")
        v = buf[16 + k:16 + k + a.size].view(a.shape)
        if not fill:
            v.copy_(torch.from_numpy(a))
        return buf, v
    mk = lambda t: ie.Mat(at(t.mant)[1], at(t.exp)[1], t.group)  # noqa: E731
    for yg in (T, R):
        (bm, vm), (be, ve) = at(D.mant, True), at(np.zeros(M if yg == R else 1, np.int8), True)
        Y = ie.Mat(vm, ve, yg)
        ie.ie_linear_fwd_fused(qt_to_dev(X), qt_to_dev(W), mk(b), mk(D), Y, ie.ACT_RELU, ws)
        assert_same(Y, o.linear_fwd_fused(X, W, b, D, yg, True), str(shape))
        for buf, n in ((bm, M * N), (be, ve.numel())):
            assert bool((buf[:16 + k] == 77).all()) and bool((buf[16 + k + n:] == 77).all())


def test_linear_fused_exponent_range_is_flagged(ws):
    announce("linear fused exponent range")
    rng = np.random.default_rng(5)
    X, W = rand_qt(rng, (66, 64), R, -6, -6), rand_qt(rng, (140, 64), R, -6, -6)
    D = o.QT(np.full((66, 140), 127, np.int8), np.full(66, 127, np.int8), R)
    X2 = o.QT(X.mant, np.full(66, 100, np.int8), R)
    W2 = o.QT(W.mant, np.full(140, 30, np.int8), R)
    for yg in (T, R):
        for x, w, d in ((X2, W2, None), (X2, W2, D)):
            bias = vec(rng, 140, R)
            ie.ie_linear_fwd_fused(qt_to_dev(x), qt_to_dev(w), dev(bias), dev(d), ie.Mat.empty(66, 140, yg), 0, ws)
            assert ws.status() == ie.FLAG_EXP_RANGE and ws.status() == 0


def test_linear_fused_stream_and_graph():
    announce("linear fused stream and graph")
    rng = np.random.default_rng(6)
    cases = []
    own = ie.Workspace("cuda")
    for M, N, K, yg in ((300, 200, 64, R), (300, 200, 64, T), (4, 100, 2048, T), (4, 100, 2048, R)):
        W, b = rand_qt(rng, (N, K), R), vec(rng, N, R)
        cases.append((M, N, K, yg, W, b, qt_to_dev(W), dev(b), ie.Mat.empty(M, K, R), ie.Mat.empty(M, N, R),
                      ie.Mat.empty(M, N, yg)))
    for c in cases:
        for m in c[8:10]:
            m.mant.zero_()
            m.exp.zero_()

    def run():
        for _, _, _, _, _, _, Wd, bd, Xd, Dd, Y in cases:
            ie.ie_linear_fwd_fused(Xd, Wd, bd, Dd, Y, ie.ACT_RELU, own)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        run()
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(3):
        hosts = []
        for M, N, K, yg, W, b, Wd, bd, Xd, Dd, Y in cases:
            X, D = rand_qt(rng, (M, K), R), rand_qt(rng, (M, N), R, -10, 2)
            hosts.append((X, D))
            for d, h in ((Xd, X), (Dd, D)):
                d.mant.copy_(torch.from_numpy(h.mant))
                d.exp.copy_(torch.from_numpy(h.exp))
        graph.replay()
        torch.cuda.synchronize()
        for (X, D), (M, N, K, yg, W, b, *_, Y) in zip(hosts, cases):
            assert_same(Y, o.linear_fwd_fused(X, W, b, D, yg, True), f"replay {i}")
    assert own.status() == 0


# (M, N, K) whose rows lie whole in a workgroup: 1..4 blocks of 256 columns,
# short and staged contractions (K over 1024 in two stages), one and several
# tiles to a workgroup, the last one ragged
ROWS = [(2048, 129, 16), (2049, 256, 1040), (33000, 130, 40), (6145, 300, 1030), (2063, 511, 256), (16500, 512, 33),
        (6160, 520, 300), (17001, 768, 96), (2100, 770, 192), (6144, 1000, 2048), (16449, 1024, 130)]


@pytest.mark.parametrize("shape", ROWS, ids=lambda s: "x".join(map(str, s)))
def test_linear_fused_many_rows(shape, ws):
    M, N, K = shape
    announce(f"linear fused rows {shape}")
    rng = np.random.default_rng(M + N + K)
    for xg, wg, dg, relu, some in ((R, R, R, True, 3), (T, R, T, False, 3), (R, T, R, False, 2), (T, T, T, True, 1)):
        X, W = rand_qt(rng, (M, K), xg), rand_qt(rng, (N, K), wg)
        X.mant[M // 2] = 0
        b = vec(rng, N, R if some == 3 else T) if some & 1 else None
        D = rand_qt(rng, (M, N), dg, -10, 2) if some & 2 else None
        check(X, W, b, D, R, relu, ws, bits=8 if some & 1 else 5, what=f"{shape} {some}")


@pytest.mark.parametrize("gap", [-120, -60, -25, 0, 25, 60, 120])
@pytest.mark.parametrize("shape", [(2070, 140, 64), (2050, 900, 48)], ids=lambda s: "x".join(map(str, s)))
def test_linear_fused_many_rows_far_exponents(gap, shape, ws):
    announce(f"linear fused rows gap {gap} {shape}")
    M, N, K = shape
    rng = np.random.default_rng(gap + 300)
    X, W = rand_qt(rng, (M, K), R, -6, -6), rand_qt(rng, (N, K), R, -6, -6)
    X.mant[1], W.mant[2], X.mant[3], W.mant[3] = 0, 0, -128, -128
    e = np.clip(-12 + gap, -128, 110)
    b = o.QT(rng.integers(-128, 128, (N, 1)).astype(np.int8), np.full(N, e, np.int8), R)
    b.mant[::3] = 0
    D = o.QT(rng.integers(-128, 128, (M, N)).astype(np.int8), np.full(M, np.clip(-12 - gap, -128, 110), np.int8), R)
    D.mant[1], D.mant[:, 5] = 0, 0
    for bb, dd in ((b, D), (b, None), (None, D)):
        check(X, W, bb, dd, R, False, ws, what=f"gap {gap}")


@pytest.mark.parametrize("k", [0, 1, 2, 8])
@pytest.mark.parametrize("shape", [(2070, 208, 64), (2070, 323, 32), (17000, 528, 80)],
                         ids=lambda s: "x".join(map(str, s)))
def test_linear_fused_many_rows_guards(k, shape, ws):
    """Residual, bias and result at odd addresses; nothing written beside the result."""
    announce(f"linear fused rows {shape} off by {k}")
    M, N, K = shape
    rng = np.random.default_rng(k)
    X, W = rand_qt(rng, (M, K), R), rand_qt(rng, (N, K), R)
    b, D = vec(rng, N, R), rand_qt(rng, (M, N), R, -10, 2)

    def at(a, fill=False):
        buf = torch.full((a.size + 64,), 77, dtype=torch.int8, device="cuda")
        v = buf[16 + k:16 + k + a.size].view(a.shape)
        if not fill:
            v.copy_(torch.from_numpy(a))
        return buf, v
    mk = lambda t: ie.Mat(at(t.mant)[1], at(t.exp)[1], t.group)  # noqa: E731
    (bm, vm), (be, ve) = at(D.mant, True), at(np.zeros(M, np.int8), True)
    ie.ie_linear_fwd_fused(qt_to_dev(X), qt_to_dev(W), mk(b), mk(D), ie.Mat(vm, ve, R), ie.ACT_RELU, ws)
    assert_same(ie.Mat(vm, ve, R), o.linear_fwd_fused(X, W, b, D, R, True), str(shape))
    for buf, n in ((bm, M * N), (be, M)):
        assert bool((buf[:16 + k] == 77).all()) and bool((buf[16 + k + n:] == 77).all())


def test_linear_fused_many_rows_flag_and_graph():
    """The exponent-range flag, then replays on new inputs, eager work between them."""
    announce("linear fused rows flag and graph")
    rng = np.random.default_rng(8)
    own = ie.Workspace("cuda")
    M, N, K = 2100, 200, 64
    W, b = rand_qt(rng, (N, K), R), vec(rng, N, R)
    Wd, bd = qt_to_dev(W), dev(b)
    Xd, Dd, Y = ie.Mat.empty(M, K, R), ie.Mat.empty(M, N, R), ie.Mat.empty(M, N, R)
    X, D = rand_qt(rng, (M, K), R, 126, 127), rand_qt(rng, (M, N), R)

    def put():
        for d, h in ((Xd, X), (Dd, D)):
            d.mant.copy_(torch.from_numpy(h.mant))
            d.exp.copy_(torch.from_numpy(h.exp))

    def run():
        ie.ie_linear_fwd_fused(Xd, Wd, bd, Dd, Y, ie.ACT_NONE, own)
    put()
    W2 = qt_to_dev(o.QT(W.mant, np.full(N, 30, np.int8), R))
    ie.ie_linear_fwd_fused(Xd, W2, bd, Dd, Y, ie.ACT_NONE, own)
    assert own.status() == ie.FLAG_EXP_RANGE and own.status() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
        run()
    for i in range(3):
        X, D = rand_qt(rng, (M, K), R), rand_qt(rng, (M, N), R, -10, 2)
        put()
        graph.replay()
        assert_same(Y, o.linear_fwd_fused(X, W, b, D, R), f"replay {i}")
        check(X, W, b, D, R, True, own)
    assert own.status() == 0


# up to 64 rows: 1, 2 and 4 blocks of 16, short and long contractions, columns
# off the blocks of 16 and the runs of 4, contractions off the runs of 16;
# beside them single tiles and splits over several rows
FEW = [(1, 65, 16), (1, 4096, 4096), (2, 130, 1024), (16, 257, 1025), (17, 300, 2000), (32, 1030, 17), (33, 77, 2064),
       (64, 129, 63), (64, 1000, 1500), (5, 4099, 4100), (3, 2050, 65536), (16, 16000, 48), (65, 66, 256),
       (128, 128, 200), (6, 60, 2048), (70, 200, 2048), (100, 333, 1039)]


@pytest.mark.parametrize("shape", FEW, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("yg", [T, R])
def test_linear_fused_few_rows(shape, yg, ws):
    M, N, K = shape
    announce(f"linear fused few rows {shape} {yg}")
    rng = np.random.default_rng(M + N + K)
    for xg, wg, dg, some in ((R, R, R, 3), (T, R, T, 2), (R, T, R, 1), (T, T, T, 3)):
        X, W = rand_qt(rng, (M, K), xg), rand_qt(rng, (N, K), wg)
        X.mant[M // 2] = 0
        b = vec(rng, N, R if some == 3 else T) if some & 1 else None
        D = rand_qt(rng, (M, N), dg, -10, 2) if some & 2 else None
        check(X, W, b, D, yg, some == 3, ws, bits=8 if some & 1 else 5, what=f"{shape} {some}")


@pytest.mark.parametrize("gap", [-120, -60, -25, 0, 25, 60, 120])
@pytest.mark.parametrize("shape", [(9, 140, 64), (40, 131, 2048), (6, 60, 2048), (70, 130, 128)],
                         ids=lambda s: "x".join(map(str, s)))
def test_linear_fused_few_rows_far_exponents(gap, shape, ws):
    announce(f"linear fused few rows gap {gap} {shape}")
    M, N, K = shape
    rng = np.random.default_rng(gap + 400)
    X, W = rand_qt(rng, (M, K), R, -6, -6), rand_qt(rng, (N, K), R, -6, -6)
    X.mant[1], W.mant[2], X.mant[3], W.mant[3] = 0, 0, -128, -128
    e = np.clip(-12 + gap, -128, 110)
    b = o.QT(rng.integers(-128, 128, (N, 1)).astype(np.int8), np.full(N, e, np.int8), R)
    b.mant[::3] = 0
    D = o.QT(rng.integers(-128, 128, (M, N)).astype(np.int8), np.full(M, np.clip(-12 - gap, -128, 110), np.int8), R)
    D.mant[1], D.mant[:, 5] = 0, 0
    for yg, bb, dd in ((R, b, D), (T, b, D), (R, b, None), (T, None, D)):
        check(X, W, bb, dd, yg, False, ws, what=f"gap {gap}")


@pytest.mark.parametrize("k", [0, 1, 4])
@pytest.mark.parametrize("shape", [(3, 131, 48), (50, 272, 1200), (7, 31, 2048)], ids=lambda s: "x".join(map(str, s)))
def test_linear_fused_few_rows_guards(k, shape, ws):
    """Residual, bias and result at odd addresses; nothing written beside the result."""
    announce(f"linear fused few rows {shape} off by {k}")
    M, N, K = shape
    rng = np.random.default_rng(k)
    X, W = rand_qt(rng, (M, K), R), rand_qt(rng, (N, K), R)
    b, D = vec(rng, N, R), rand_qt(rng, (M, N), R, -10, 2)

    def at(a, fill=False):
        buf = torch.full((a.size + 64,), 77, dtype=torch.int8, device="cuda")
        v = buf[16 + k:16 + k + a.size].view(a.shape)
        if not fill:
            v.copy_(torch.from_numpy(a))
        return buf, v
    mk = lambda t: ie.Mat(at(t.mant)[1], at(t.exp)[1], t.group)  # noqa: E731
    for yg in (T, R):
        (bm, vm), (be, ve) = at(D.mant, True), at(np.zeros(M if yg == R else 1, np.int8), True)
        ie.ie_linear_fwd_fused(qt_to_dev(X), qt_to_dev(W), mk(b), mk(D), ie.Mat(vm, ve, yg), ie.ACT_RELU, ws)
        assert_same(ie.Mat(vm, ve, yg), o.linear_fwd_fused(X, W, b, D, yg, True), str(shape))
        for buf, n in ((bm, M * N), (be, ve.numel())):
            assert bool((buf[:16 + k] == 77).all()) and bool((buf[16 + k + n:] == 77).all())


@pytest.mark.parametrize("yg", [T, R])
def test_linear_fused_few_rows_flag_and_graph(yg):
    """The exponent-range flag, then replays on new inputs, eager work between them."""
    announce(f"linear fused few rows flag and graph {yg}")
    rng = np.random.default_rng(9)
    own = ie.Workspace("cuda")
    M, N, K = 4, 200, 64
    W, b = rand_qt(rng, (N, K), R), vec(rng, N, R)
    Wd, bd = qt_to_dev(W), dev(b)
    Xd, Dd, Y = ie.Mat.empty(M, K, R), ie.Mat.empty(M, N, R), ie.Mat.empty(M, N, yg)
    X, D = rand_qt(rng, (M, K), R, 126, 127), rand_qt(rng, (M, N), R)

    def put():
        for d, h in ((Xd, X), (Dd, D)):
            d.mant.copy_(torch.from_numpy(h.mant))
            d.exp.copy_(torch.from_numpy(h.exp))
    put()
    W2 = qt_to_dev(o.QT(W.mant, np.full(N, 30, np.int8), R))
    ie.ie_linear_fwd_fused(Xd, W2, bd, Dd, Y, ie.ACT_NONE, own)
    assert own.status() == ie.FLAG_EXP_RANGE and own.status() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            ie.ie_linear_fwd_fused(Xd, Wd, bd, Dd, Y, ie.ACT_NONE, own)
    for i in range(3):
        X, D = rand_qt(rng, (M, K), R), rand_qt(rng, (M, N), R, -10, 2)
        put()
        graph.replay()
        assert_same(Y, o.linear_fwd_fused(X, W, b, D, yg), f"replay {i}")
        check(X, W, b, D, yg, True, own)
    assert own.status() == 0


@pytest.mark.parametrize("shape", [(2100, 300, 96), (2048, 257, 33), (7, 300, 77), (64, 640, 1024), (1, 33, 16)],
                         ids=lambda s: "x".join(map(str, s)))
def test_linear_fused_without_addends_in_few_and_whole_rows(shape, ws):
    announce(f"linear fused plain {shape}")
    M, N, K = shape
    rng = np.random.default_rng(11)
    for xg, wg, yg in ((R, R, R), (T, R, R), (T, T, T)):
        X, W = rand_qt(rng, (M, K), xg), rand_qt(rng, (N, K), wg)
        for act in (ie.ACT_NONE, ie.ACT_RELU):
            Y, Z = ie.Mat.empty(M, N, yg), ie.Mat.empty(M, N, yg)
            ie.ie_linear_fwd_fused(qt_to_dev(X), qt_to_dev(W), None, None, Y, act, ws)
            ie.ie_linear_fwd_act(qt_to_dev(X), qt_to_dev(W), Z, act, ws)
            torch.cuda.synchronize()
            assert torch.equal(Y.mant, Z.mant) and torch.equal(Y.exp, Z.exp)
    assert ws.status() == 0


# contractions split over workgroups, and one tile's few rows that are not
SPLIT = [(16, 80, 4096), (70, 130, 1100), (40, 70, 4000), (17, 40, 4096), (16, 64, 9000), (5, 1, 7747), (1, 7, 65536)]


@pytest.mark.parametrize("shape", SPLIT, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("yg", [T, R])
def test_linear_fused_long_contractions(shape, yg, ws):
    announce(f"linear fused long {shape} {yg}")
    M, N, K = shape
    rng = np.random.default_rng(M + N + K)
    X, W = rand_qt(rng, (M, K), R), rand_qt(rng, (N, K), R)
    b, D = vec(rng, N, R), rand_qt(rng, (M, N), R, -10, 2)
    for relu, bb, dd in ((True, b, D), (False, b, None), (False, None, D)):
        check(X, W, bb, dd, yg, relu, ws, what=f"{shape}")


@pytest.mark.parametrize("shape", [(300, 1027, 65), (130, 90, 300), (2500, 1100, 48), (400, 1033, 1040)],
                         ids=lambda s: "x".join(map(str, s)))
def test_linear_fused_without_addends_off_the_runs(shape, ws):
    announce(f"linear fused plain {shape}")
    M, N, K = shape
    rng = np.random.default_rng(12)
    for xg, wg, yg in ((R, R, R), (T, T, T)):
        X, W = rand_qt(rng, (M, K), xg), rand_qt(rng, (N, K), wg)
        for act in (ie.ACT_NONE, ie.ACT_RELU):
            Y, Z = ie.Mat.empty(M, N, yg), ie.Mat.empty(M, N, yg)
            ie.ie_linear_fwd_fused(qt_to_dev(X), qt_to_dev(W), None, None, Y, act, ws)
            ie.ie_linear_fwd_act(qt_to_dev(X), qt_to_dev(W), Z, act, ws)
            torch.cuda.synchronize()
            assert torch.equal(Y.mant, Z.mant) and torch.equal(Y.exp, Z.exp)
    assert ws.status() == 0
