"""ie_attention_cache over contexts of many blocks, against the oracle bit for bit: the joining of the blocks' sums."""

import numpy as np
import pytest
import torch

import oracle as o
from integer_only_dnn_amd import ie
from tests.attention_util import dev_i32, filled, qkv
from tests.gpu_util import announce, assert_same, from_dev, qt_to_dev

pytestmark = pytest.mark.gpu


def cache_of(k, v, ke, ve):
    """(host, device) from mantissas [pages, page, kv, d] and exponents [pages, page, kv]."""
    pages, page, kv, d = k.shape
    host = dict(k=o.pack4(k).reshape(pages * page, kv, d // 2), v=o.pack4(v).reshape(pages * page, kv, d // 2),
                ke=ke.astype(np.int8).reshape(-1, kv), ve=ve.astype(np.int8).reshape(-1, kv))
    dev = [torch.from_numpy(host[z].reshape(pages, page, kv, -1).copy()).cuda() for z in ("k", "v")]
    exps = [torch.from_numpy(host[z].reshape(pages, page, kv).copy()).cuda() for z in ("ke", "ve")]
    return host, ie.Cache(dev[0], exps[0], dev[1], exps[1])


def attend(host, cache, Q, table, lengths, heads, kv, d, scale, rows=None):
    """The call, and the oracle's result of some of its rows (None: all)."""
    page = cache.desc.page
    ws, O = ie.Workspace("cuda"), filled(len(lengths), heads * d)
    ie.ie_attention_cache(ie.Attention(heads, kv, d, scale), qt_to_dev(Q), cache, dev_i32(table), dev_i32(lengths), O, ws)
    rows = range(len(lengths)) if rows is None else rows
    slots = [table[i][np.arange(lengths[i]) // page] * page + np.arange(lengths[i]) % page for i in rows]
    want = o.attention_cache(o.QT(Q.mant[rows], Q.exp[rows], o.ROW), host, slots, heads, kv, d, scale)
    assert ws.status() == 0
    return O, want


def test_largest_context():
    """2^23 positions of one page, all scores alike, all values 7 (or -8): the largest sums there are."""
    announce("cache join 2^23 positions")
    page, per, d = 256, 1 << 15, 16
    v = np.full((1, page, 1, d), 7)
    v[..., 1] = -8
    host, cache = cache_of(np.ones((1, page, 1, d)), v, np.zeros((1, page, 1)), np.zeros((1, page, 1)))
    Q = o.QT(np.zeros((1, d), np.int8), np.array([-8], np.int8), o.ROW)
    O, want = attend(host, cache, Q, np.zeros((1, per), np.int64), [page * per], 1, 1, d, 0.25)
    assert_same(O, want, "O")
    # 7 and -8 themselves: 8 is 64 2^-3, and 128 2^-4 would be too much
    assert from_dev(O)[1][0] == -3 and list(from_dev(O)[0][0, :2]) == [56, -64]


@pytest.mark.parametrize("n,heads,d", [(1, 1, 16), (1, 4, 64), (520, 1, 16), (2, 260, 16)])
def test_many_blocks_of_values_that_cancel(n, heads, d):
    """A million positions: values of one sign in half of the blocks, of the other sign in the rest, weights near one; one
    sequence among few and among many, where the elements of a head are shared out otherwise."""
    announce(f"cache join cancelling {n} {heads} {d}")
    rng = np.random.default_rng(5)
    page, pages = 256, 64
    k, v = rng.integers(-1, 2, (pages, page, 1, d)), rng.integers(0, 8, (pages, page, 1, d))
    v[1::2] = -v[0::2]
    v[-1] = rng.integers(-7, 8, v[-1].shape)
    k[1::2] = k[0::2]
    host, cache = cache_of(k, v, np.full((pages, page, 1), -3), np.full((pages, page, 1), 0))
    per = 4096 if n * heads == 1 else 1024
    table = np.concatenate([np.tile(np.arange(0, pages, 2), per // 64), np.tile(np.arange(1, pages, 2), per // 64)])[None].repeat(n, 0)
    lengths = [per * page] + [300 + i for i in range(n - 1)]
    Q = qkv(rng, n, heads, 0, d, elo=-9, ehi=-8)
    Q.mant[:1] = np.tile(Q.mant[:1, :d], (1, heads))
    O, want = attend(host, cache, Q, table, lengths, heads, 1, d, float(np.float32(d ** -0.5)), rows=[0, n - 1] if n > 1 else [0])
    m, e = from_dev(O)
    for at, row in enumerate([0, n - 1] if n > 1 else [0]):
        assert e[row] == want.exp[at] and np.array_equal(m[row], want.mant[at]), row


def sinks(rng, n, gap, heads, kv, d, page, spread):
    """A cache whose first key is `gap` nats ahead of the others for every head, its value zero; pages out of order."""
    pages = -(-n // page) + 2
    k, v = rng.integers(-1, 2, (pages, page, kv, d)), np.clip(np.rint(rng.normal(1, 3, (pages, page, kv, d))), -7, 7).astype(int)
    k[..., 0] = 0
    order = rng.permutation(pages)[:-(-n // page)]
    ke, ve = np.full((pages, page, kv), -6), rng.integers(-2 - spread, -1, (pages, page, kv))
    k[order[0], 0], v[order[0], 0] = 0, 0
    k[order[0], 0, :, 0] = 7
    ke[order[0], 0], ve[order[0], 0] = 0, -128
    Q = rng.integers(-60, 61, (1, heads, d))
    Q[:, :, 0] = 100
    return cache_of(k, v, ke, ve), order, o.QT(Q.reshape(1, -1).astype(np.int8), np.array([-8], np.int8), o.ROW), gap / (7 * 100 / 256)


@pytest.mark.parametrize("n,gap,heads,kv,d,page,spread", [(2305, 11.5, 1, 1, 16, 16, 0), (4000, 10.5, 4, 2, 64, 64, 2), (70000, 12.0, 2, 2, 32, 256, 4),
                                                          (131072, 13.0, 4, 1, 128, 256, 0), (9000, 11.0, 3, 3, 48, 1, 1)])
def test_sinks(n, gap, heads, kv, d, page, spread):
    announce(f"cache tail {n} {gap} {heads} {kv} {d}")
    (host, cache), order, Q, scale = sinks(np.random.default_rng(n), n, gap, heads, kv, d, page, spread)
    O, want = attend(host, cache, Q, order[None], [n], heads, kv, d, float(np.float32(scale)))
    assert_same(O, want, "O")


def test_sinks_among_others():
    """More heads than a workgroup's shares: whole heads to a workgroup; sequences with and without a sink, short and empty ones."""
    announce("cache tail batch")
    rng = np.random.default_rng(3)
    (host, cache), order, Q, scale = sinks(rng, 3000, 11.0, 4, 2, 32, 16, 1)
    n = 140
    lengths = rng.integers(0, 2900, n)
    lengths[:4] = [3000, 0, 2049, 2048]
    table = np.tile(order, (n, 1))
    for i in range(5, n, 2):
        table[i] = np.roll(order, -1)  # no sink
    X = qkv(rng, n, 4, 0, 32, elo=-8, ehi=-8)
    X.mant[:] = Q.mant
    X.mant[6::4] //= 8
    rows = [0, 1, 2, 3, 4, 5, 6, 7, 10, 139]
    O, want = attend(host, cache, X, table, [int(t) for t in lengths], 4, 2, 32, float(np.float32(scale)), rows)
    m, e = from_dev(O)
    for at, row in enumerate(rows):
        assert e[row] == want.exp[at] and np.array_equal(m[row], want.mant[at]), row
