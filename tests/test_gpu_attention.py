"""ie_attention_fwd and ie_attention_bwd against the oracle, bit for bit: head layouts and sizes, lengths around every
tile's edge, packed and empty sequences, extreme exponents, strides and widths."""

import numpy as np
import pytest
import torch

import oracle as o
from integer_only_dnn_amd import ie
from tests.attention_util import (assert_rows, dev_i32, filled, offsets_of, qkv, shifted, stats_of, to_dev)
from tests.gpu_util import announce, rand_qt

pytestmark = pytest.mark.gpu


def run(X, heads, kv, d, causal, offsets, scale=None, bits=8, dO=None, by=0, spoil=True):
    """Forward (with stats) and, with dO, backward; both compared with the oracle."""
    rows = X.mant.shape[0]
    scale = float(np.float32(d ** -0.5)) if scale is None else scale
    ws = ie.Workspace("cuda")
    ws.get(1 << 16)
    if spoil:
        ws.buf[256:].fill_(0x5a)  # nothing in a workspace starts at any value
    att = ie.Attention(heads, kv, d, scale, causal, None if offsets is None else dev_i32(offsets))
    Xd = shifted(X, by) if by else to_dev(X)
    O, stats = filled(rows, heads * d, bits, by), stats_of(rows, heads)
    ie.ie_attention_fwd(att, Xd, O, ws, stats)
    want, m, L = o.attention_fwd(X, heads, kv, d, scale, causal, offsets, bits)
    covered = (0, rows) if offsets is None else (offsets[0], offsets[-1])
    assert_rows(O, want, covered, "O")
    got = stats.cpu().numpy()[covered[0]:covered[1]]
    assert np.array_equal(got[..., 0].view(np.float32), m[covered[0]:covered[1]])
    assert np.array_equal(got[..., 1], L[covered[0]:covered[1]])
    O2 = filled(rows, heads * d, bits, by)
    ie.ie_attention_fwd(att, Xd, O2, ws)
    assert_rows(O2, want, covered, "O without stats")
    if dO is not None:
        G = filled(rows, (heads + 2 * kv) * d, bits, by)
        ie.ie_attention_bwd(att, Xd, O, shifted(dO, by) if by else to_dev(dO), stats, G, ws)
        wantG = o.attention_bwd(X, want, dO, m, L, heads, kv, d, scale, causal, offsets, bits)
        assert_rows(G, wantG, covered, "dQKV")
    assert ws.status() == 0
    return want


LENGTHS = [[1], [2], [31], [32], [33], [63, 64, 65], [127], [128], [129], [197, 1, 0, 0, 300], [0], [260, 5]]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("group", [o.ROW, o.TENSOR])
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda v: "+".join(map(str, v)))
def test_lengths(lengths, group, causal):
    announce(f"attention lengths {lengths} {group} {causal}")
    rng = np.random.default_rng(sum(lengths) + 7 * causal)
    heads, kv, d = 4, 2, 32
    rows = sum(lengths) + 5  # two rows in front of the first sequence, three behind the last
    X = qkv(rng, rows, heads, kv, d, group)
    run(X, heads, kv, d, causal, offsets_of(lengths, 2), dO=rand_qt(rng, (rows, heads * d), group, -20, -14))


@pytest.mark.parametrize("heads,kv,d", [(1, 1, 1), (2, 1, 2), (3, 3, 7), (1, 1, 16), (5, 1, 20), (4, 4, 31), (2, 2, 33), (6, 2, 40),
                                        (2, 1, 48), (3, 3, 64), (2, 2, 65), (4, 1, 80), (2, 1, 96), (3, 1, 100), (2, 2, 112),
                                        (8, 2, 128), (17, 1, 32), (70, 70, 4)])
@pytest.mark.parametrize("causal", [False, True])
def test_heads(heads, kv, d, causal):
    announce(f"attention heads {heads} {kv} {d} {causal}")
    rng = np.random.default_rng(heads * 131 + d)
    X = qkv(rng, 143, heads, kv, d)
    run(X, heads, kv, d, causal, [0, 70, 143], dO=rand_qt(rng, (143, heads * d), o.ROW, -12, -9))


@pytest.mark.parametrize("by", [1, 4, 8, 16])
@pytest.mark.parametrize("d", [32, 36])
def test_alignment(by, d):
    announce(f"attention {by} bytes off, {d}")
    rng = np.random.default_rng(by + d)
    X = qkv(rng, 90, 4, 2, d)
    run(X, 4, 2, d, True, [0, 90], dO=rand_qt(rng, (90, 4 * d), o.ROW, -12, -9), by=by)


@pytest.mark.parametrize("bits", [2, 4, 7])
def test_widths(bits):
    announce(f"attention into {bits} bits")
    rng = np.random.default_rng(bits)
    X = qkv(rng, 75, 2, 1, 64)
    run(X, 2, 1, 64, True, None, bits=bits, dO=rand_qt(rng, (75, 128), o.TENSOR))


@pytest.mark.parametrize("scale", [2.0 ** -30, 1.0, 37.5, 2.0 ** 30])
@pytest.mark.parametrize("exps", [(-9, -5), (-60, -40), (-128, -100), (8, 16), (-48, 16), (-128, 16)])
def test_scales_and_exponents(scale, exps):
    """Weights from all alike to a single one, exponents at and past the clipping, far apart within a sequence."""
    announce(f"attention scale {scale} exponents {exps}")
    rng = np.random.default_rng(int(abs(np.log2(scale))) + exps[0] + 200)
    for causal in (False, True):
        X = qkv(rng, 70, 2, 1, 32, o.ROW, *exps, flat=True)
        run(X, 2, 1, 32, causal, [0, 1, 70], scale=float(scale), dO=rand_qt(rng, (70, 64), o.ROW, -128, 20))


def test_zero_rows_and_extreme_mantissas():
    """Padding rows (all zero, exponent -128), all mantissas -128, gradients of zeros."""
    announce("attention zero rows")
    rng = np.random.default_rng(1)
    X = qkv(rng, 100, 2, 2, 64)
    X.mant[10:20], X.exp[10:20] = 0, -128
    X.mant[40:60] = -128
    dO = rand_qt(rng, (100, 128), o.ROW, -12, -9)
    dO.mant[30:50], dO.exp[30:50] = 0, -128
    for causal in (False, True):
        run(X, 2, 2, 64, causal, [0, 33, 100], dO=dO)
    Z = o.QT(np.zeros((40, 3 * 32), np.int8), np.full(40, -128, np.int8), o.ROW)
    run(Z, 1, 1, 32, True, None, dO=o.QT(np.zeros((40, 32), np.int8), np.full(40, -128, np.int8), o.ROW))
    A = o.QT(np.full((140, 3 * 128), -128, np.int8), np.array([3], np.int8), o.TENSOR)
    run(A, 1, 1, 128, False, None, dO=o.QT(np.full((140, 128), -128, np.int8), np.array([0], np.int8), o.TENSOR))


def test_many_short_sequences():
    announce("attention many sequences")
    rng = np.random.default_rng(5)
    lengths = rng.integers(0, 9, 700)
    rows = int(lengths.sum())
    X = qkv(rng, rows, 2, 1, 16)
    run(X, 2, 1, 16, True, offsets_of(lengths), dO=rand_qt(rng, (rows, 32), o.ROW, -12, -9))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("heads,kv,d,lengths", [(128, 64, 16, [300]), (256, 256, 4, [300]), (130, 2, 128, [290]),
                                                (8, 8, 64, [280] + 200 * [1]), (8, 8, 128, [1, 259] + 220 * [1]),
                                                (8, 8, 96, 200 * [2] + [257]), (9, 9, 32, 130 * [0, 3] + [333]),
                                                (40, 40, 70, [150, 70]), (80, 40, 101, [121, 0, 100])],
                         ids=lambda v: "+".join(map(str, v[:2])) + f"_{len(v)}" if isinstance(v, list) else str(v))
def test_full_grids(heads, kv, d, lengths, causal):
    """Tiles enough that no launch splits a tile's keys or queries over its waves."""
    announce(f"attention full grids {heads} {kv} {d} {len(lengths)} {causal}")
    rng = np.random.default_rng(heads + d)
    rows = sum(lengths)
    X = qkv(rng, rows, heads, kv, d, o.TENSOR if d == 4 else o.ROW)
    run(X, heads, kv, d, causal, offsets_of(lengths), dO=rand_qt(rng, (rows, heads * d), o.ROW, -12, -9))


def test_sequences_in_chunks():
    """So many tiles that an XCD takes several chunks of them, the last one smaller."""
    announce("attention chunks")
    rng = np.random.default_rng(8)
    lengths = rng.integers(0, 70, 333)
    rows = int(lengths.sum())
    X = qkv(rng, rows, 3, 1, 16)
    run(X, 3, 1, 16, False, offsets_of(lengths), dO=rand_qt(rng, (rows, 48), o.ROW, -12, -9))


@pytest.mark.parametrize("causal", [False, True])
def test_long(causal):
    """Past 1024 keys: several turns of every loop; a peaked row beside flat ones."""
    announce(f"attention long {causal}")
    rng = np.random.default_rng(11)
    X = qkv(rng, 1500, 2, 1, 64)
    X.mant[700:710] = np.clip(X.mant[700:710].astype(int) * 3, -127, 127)
    run(X, 2, 1, 64, causal, [0, 1111, 1500], dO=rand_qt(rng, (1500, 128), o.ROW, -12, -9))


def test_offsets_that_lie_outside():
    """Offsets past the matrix, negative or falling set the flag; nothing else is written."""
    announce("attention bad offsets")
    rng = np.random.default_rng(3)
    X = qkv(rng, 64, 2, 1, 32)
    Xd, ws = to_dev(X), ie.Workspace("cuda")
    for bad in ([0, 10, 1 << 30], [-5, 10, 20], [0, 40, 30, 64], [70, 80]):
        att = ie.Attention(2, 1, 32, 0.25, True, dev_i32(bad))
        guard = torch.full((64 * 64 + 4096,), 77, dtype=torch.int8, device="cuda")
        O = ie.Mat(guard[2048:2048 + 64 * 64].view(64, 64), torch.full((64,), 77, dtype=torch.int8, device="cuda"), ie.ROW)
        stats = stats_of(64, 2)
        ie.ie_attention_fwd(att, Xd, O, ws, stats)
        assert ws.status() == ie.FLAG_INDEX
        G = filled(64, 128)
        ie.ie_attention_bwd(att, Xd, O, to_dev(rand_qt(rng, (64, 64), o.ROW)), stats, G, ws)
        assert ws.status() == ie.FLAG_INDEX
        g = guard.cpu().numpy()
        assert np.all(g[:2048] == 77) and np.all(g[2048 + 4096:] == 77)


def test_large_exponents_are_flagged():
    announce("attention exponent flag")
    rng = np.random.default_rng(4)
    X = qkv(rng, 40, 1, 1, 32)
    X.exp[39] = 17
    ws, O, stats = ie.Workspace("cuda"), filled(40, 32), stats_of(40, 1)
    att = ie.Attention(1, 1, 32, 0.25, True)
    ie.ie_attention_fwd(att, to_dev(X), O, ws, stats)
    assert ws.status() == ie.FLAG_EXP_RANGE
    # causal: the rows before it do not depend on it
    want = o.attention_fwd(o.QT(X.mant[:39], X.exp[:39], o.ROW), 1, 1, 32, 0.25, True)[0]
    m, e = O.mant.cpu().numpy(), O.exp.cpu().numpy()
    assert np.array_equal(m[:39], want.mant) and np.array_equal(e[:39], want.exp)
