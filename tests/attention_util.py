"""Inputs and comparisons shared by the GPU tests of attention, rotary positions and the 4-bit cache."""

import numpy as np
import torch

import oracle as o
from integer_only_dnn_amd import ie
from tests.gpu_util import from_dev, qt_to_dev, rand_qt

SENTINEL = 77


def offsets_of(lengths, first=0):
    return [first] + [first + int(t) for t in np.cumsum(lengths)]


def dev_i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def shifted(t: o.QT, by: int) -> ie.Mat:
    """A device matrix whose mantissas start `by` bytes behind an aligned address."""
    m = np.ascontiguousarray(t.mant)
    buf = torch.zeros(m.size + 64, dtype=torch.int8, device="cuda")
    view = buf[by:by + m.size].view(m.shape)
    view.copy_(torch.from_numpy(m))
    return ie.Mat(view, torch.from_numpy(np.asarray(t.exp, dtype=np.int8).copy()).cuda(), t.group)


def filled(rows, cols, bits=8, by=0):
    """An output matrix with one exponent a row, full of a value that must stay where nothing is written."""
    buf = torch.full((rows * cols + 64,), SENTINEL, dtype=torch.int8, device="cuda")
    return ie.Mat(buf[by:by + rows * cols].view(rows, cols), torch.full((rows,), SENTINEL, dtype=torch.int8, device="cuda"), ie.ROW,
                  bits)


def assert_rows(got: ie.Mat, want: o.QT, covered, what=""):
    """Rows of sequences equal the oracle's, all others are as they were."""
    m, e = from_dev(got)
    inside = np.zeros(len(e), bool)
    inside[covered[0]:covered[1]] = True
    bad = np.flatnonzero((e != np.where(inside, want.exp, SENTINEL)) | (m != np.where(inside[:, None], want.mant, SENTINEL)).any(axis=1))
    if len(bad):
        r = int(bad[0])
        c = np.flatnonzero(m[r] != want.mant[r])
        raise AssertionError(f"{what}: {len(bad)} rows differ, first {r}: exponent {e[r]} want {want.exp[r]}, "
                             f"columns {c[:8]} got {m[r][c[:8]]} want {want.mant[r][c[:8]]}")


def qkv(rng, rows, heads, kv, d, group=o.ROW, elo=-9, ehi=-5, flat=False):
    X = rand_qt(rng, (rows, (heads + 2 * kv) * d), group, elo, ehi)
    if not flat:
        X.mant[:] = np.clip(np.rint(rng.normal(0, 45, X.mant.shape)), -128, 127)
    return X


def stats_of(rows, heads):
    return torch.full((rows, heads, 2), SENTINEL, dtype=torch.int32, device="cuda")


def to_dev(t):
    return qt_to_dev(t)
