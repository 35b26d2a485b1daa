"""ie_rope and ie_rope_table against the oracle, bit for bit."""

import numpy as np
import pytest
import torch

import oracle as o
from integer_only_dnn_amd import ie
from tests.attention_util import dev_i32, shifted
from tests.gpu_util import announce, assert_same, qt_to_dev, rand_qt

pytestmark = pytest.mark.gpu


def run(X, heads, d, rot, interleaved, inverse, group, pos, positions, bits=8, by=0, **freq):
    rows, cols = X.mant.shape
    rope = ie.Rope(d, rot, positions, interleaved, **freq)
    ws, Y = ie.Workspace("cuda"), ie.Mat.empty(rows, cols, group, bits=bits)
    if by:
        Y = ie.Mat(torch.zeros(rows * cols + 64, dtype=torch.int8, device="cuda")[by:by + rows * cols].view(rows, cols), Y.exp, group,
                   bits)
    ie.ie_rope(rope, shifted(X, by) if by else qt_to_dev(X), None if pos is None else dev_i32(pos), Y, heads, ws, inverse)
    table = o.rope_table(o.rope_frequencies(rot, **freq), positions)
    at = np.arange(rows) if pos is None else np.asarray(pos)
    assert_same(Y, o.rope(X, at, table, heads, d, rot, interleaved, inverse, group, bits), "rope")
    assert ws.status() == 0


@pytest.mark.parametrize("rows", [1, 3, 64, 2100])
@pytest.mark.parametrize("heads,extra,d,rot", [(1, 0, 8, 8), (3, 5, 32, 32), (2, 0, 64, 32), (12, 12, 64, 64), (4, 2, 80, 40),
                                               (40, 8, 128, 128), (3, 0, 96, 16), (2, 3, 16, 0), (0, 4, 16, 8)])
def test_heads(rows, heads, extra, d, rot):
    announce(f"rope {rows} {heads} {extra} {d} {rot}")
    rng = np.random.default_rng(rows + d + rot)
    rows = rows if (heads + extra) * d * rows < 600_000 else 90
    for k, (inter, inv, gx, gy) in enumerate([(False, False, o.ROW, o.ROW), (True, True, o.ROW, o.TENSOR),
                                              (True, False, o.TENSOR, o.ROW), (False, True, o.TENSOR, o.TENSOR)]):
        X = rand_qt(rng, (rows, (heads + extra) * d), gx)
        run(X, heads, d, rot, inter, inv, gy, rng.integers(0, 300, rows), 300)


@pytest.mark.parametrize("heads,extra,d,rot", [(1, 0, 2, 2), (3, 1, 7, 6), (2, 2, 10, 10), (2, 0, 12, 4), (1, 1, 33, 32), (5, 0, 24, 20)])
def test_odd_heads(heads, extra, d, rot):
    announce(f"rope odd {heads} {d} {rot}")
    rng = np.random.default_rng(d + rot)
    for inter in (False, True):
        for group in (o.ROW, o.TENSOR):
            X = rand_qt(rng, (37, (heads + extra) * d), group)
            run(X, heads, d, rot, inter, inter, group, rng.integers(0, 50, 37), 50, bits=8 - 3 * inter)


@pytest.mark.parametrize("by", [1, 4, 8])
def test_alignment(by):
    announce(f"rope {by} bytes off")
    rng = np.random.default_rng(by)
    run(rand_qt(rng, (20, 6 * 32), o.ROW), 4, 32, 32, False, False, o.ROW, None, 20, by=by)


def test_wide_rows():
    """Rows too long to be held by a block."""
    announce("rope wide")
    rng = np.random.default_rng(6)
    for cols in (16384, 16392, 40000):
        run(rand_qt(rng, (5, cols), o.ROW), cols // 128, 128, 128, True, False, o.ROW, rng.integers(0, 9, 5), 9)
        run(rand_qt(rng, (3, cols), o.ROW), cols // 128, 128, 64, False, True, o.TENSOR, rng.integers(0, 9, 3), 9)


@pytest.mark.parametrize("exps", [(-128, -110), (100, 126), (-128, 126)])
def test_exponents(exps):
    announce(f"rope exponents {exps}")
    rng = np.random.default_rng(9)
    X = rand_qt(rng, (60, 64), o.ROW, *exps, zero_frac=0.6)
    X.mant[5] = 0
    for group in (o.ROW, o.TENSOR):
        run(X, 1, 64, 64, False, False, group, rng.integers(0, 100, 60), 100)


def test_exponent_overflow_is_flagged():
    announce("rope overflow")
    X = o.QT(np.full((2, 8), 127, np.int8), np.array([127, 0], np.int8), o.ROW)
    ws, Y = ie.Workspace("cuda"), ie.Mat.empty(2, 8, ie.ROW)
    ie.ie_rope(ie.Rope(8, 8, 2), qt_to_dev(X), dev_i32([1, 1]), Y, 1, ws)
    assert ws.status() == ie.FLAG_EXP_RANGE


@pytest.mark.parametrize("freq", [dict(), dict(factor=4.0), dict(factor=8.0, trained=8192.0), dict(base=500000.0, factor=2.5,
                                                                                              trained=100.0, low=0.5, high=32.0)])
def test_table(freq):
    """Far positions: angles in 64 bits."""
    announce(f"rope table {freq}")
    rope = ie.Rope(128, 128, 70000, **freq)
    want = o.rope_table(o.rope_frequencies(128, **freq), 70000)
    assert np.array_equal(rope.table.cpu().numpy(), want)


def test_positions_outside_the_table():
    announce("rope positions")
    rng = np.random.default_rng(8)
    X = rand_qt(rng, (6, 32), o.ROW)
    ws, Y, rope = ie.Workspace("cuda"), ie.Mat.empty(6, 32, ie.ROW), ie.Rope(32, 32, 10)
    for d, cols in ((32, 32), (16, 32)):
        for pos in ([0, 9, 10, 3, 4, 5], [0, -1, 2, 3, 4, 5], [0, 1 << 30, 2, 3, 4, -(1 << 31)]):
            ie.ie_rope(rope, qt_to_dev(X), dev_i32(pos), Y, 1, ws)
            assert ws.status() == ie.FLAG_INDEX
            at = np.where((np.array(pos) < 0) | (np.array(pos) > 9), 0, pos)
            assert_same(Y, o.rope(X, at, o.rope_table(o.rope_frequencies(32), 10), 1, 32, 32, False, False, o.ROW), "as position 0")


def test_back_again():
    """The inverse turns back, up to two roundings (half a unit each, the first one spread over a pair) and the table's."""
    announce("rope there and back")
    rng = np.random.default_rng(12)
    X = rand_qt(rng, (50, 128), o.ROW)
    rope, ws, Y, Z = ie.Rope(64, 64, 50), ie.Workspace("cuda"), ie.Mat.empty(50, 128, ie.ROW), ie.Mat.empty(50, 128, ie.ROW)
    ie.ie_rope(rope, qt_to_dev(X), None, Y, 2, ws)
    ie.ie_rope(rope, Y, None, Z, 2, ws, inverse=True)
    x = np.ldexp(X.mant.astype(float), X.exp.astype(int)[:, None])
    z = np.ldexp(Z.mant.cpu().numpy().astype(float), Z.exp.cpu().numpy().astype(int)[:, None])
    unit = np.ldexp(1.0, Y.exp.cpu().numpy().astype(int))[:, None]
    assert np.all(np.abs(z - x) <= 0.5 * 2 ** 0.5 * unit + 0.5 * np.ldexp(1.0, Z.exp.cpu().numpy().astype(int))[:, None]
                  + 8 * 2.0 ** -15 * np.abs(x).max(axis=1, keepdims=True))
