"""Attention, rotary positions and the cache where mantissas lie more than 2^32 bytes behind a matrix's or a cache's
first one, against the oracle."""

import numpy as np
import pytest
import torch

import oracle as o
from integer_only_dnn_amd import ie
from tests.attention_util import SENTINEL, dev_i32, qkv, stats_of
from tests.gpu_util import announce, assert_same, qt_to_dev, rand_qt

pytestmark = pytest.mark.gpu

HEADS, D = 30, 96
ROWS, LAST = 500_000, 400  # 4.3e9 mantissas of queries, keys and values
WIDTH = 3 * HEADS * D


@pytest.fixture(autouse=True)
def room():
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("less than 60 GiB of device memory free")
    yield
    torch.cuda.empty_cache()


def tall(cols, last: o.QT, value=0):
    """A matrix of ROWS rows, the last ones given."""
    m = torch.full((ROWS, cols), value, dtype=torch.int8, device="cuda")
    e = torch.full((ROWS,), value, dtype=torch.int8, device="cuda")
    if last is not None:
        m[-LAST:] = torch.from_numpy(last.mant).cuda()
        e[-LAST:] = torch.from_numpy(last.exp).cuda()
    return ie.Mat(m, e, ie.ROW)


def assert_last(got: ie.Mat, want: o.QT, what):
    assert bool((got.exp[:-LAST] == SENTINEL).all()) and bool((got.mant[:-LAST] == SENTINEL).all()), what
    assert np.array_equal(got.exp[-LAST:].cpu().numpy(), want.exp), what
    assert np.array_equal(got.mant[-LAST:].cpu().numpy(), want.mant), what


@pytest.mark.parametrize("causal", [False, True])
def test_attention(causal):
    announce(f"attention far {causal}")
    rng = np.random.default_rng(4)
    X, dO = qkv(rng, LAST, HEADS, HEADS, D), rand_qt(rng, (LAST, HEADS * D), o.ROW, -12, -9)
    at, scale = [0, 90, 90, LAST], float(np.float32(D ** -0.5))
    att = ie.Attention(HEADS, HEADS, D, scale, causal, dev_i32([ROWS - LAST + t for t in at]))
    Xd, O, stats, ws = tall(WIDTH, X), tall(HEADS * D, None, SENTINEL), stats_of(ROWS, HEADS), ie.Workspace("cuda")
    ie.ie_attention_fwd(att, Xd, O, ws, stats)
    want, m, L = o.attention_fwd(X, HEADS, HEADS, D, scale, causal, at)
    assert_last(O, want, "O")
    G = tall(WIDTH, None, SENTINEL)
    ie.ie_attention_bwd(att, Xd, O, tall(HEADS * D, dO), stats, G, ws)
    assert_last(G, o.attention_bwd(X, want, dO, m, L, HEADS, HEADS, D, scale, causal, at), "dQKV")
    assert ws.status() == 0


def test_rope():
    announce("rope far")
    rng = np.random.default_rng(5)
    X = rand_qt(rng, (LAST, WIDTH), o.ROW)
    Xd, Y, ws = tall(WIDTH, X), ie.Mat.empty(ROWS, WIDTH, ie.ROW), ie.Workspace("cuda")
    pos = rng.integers(0, 5000, LAST)
    posd = torch.zeros(ROWS, dtype=torch.int32, device="cuda")
    posd[-LAST:] = dev_i32(pos)
    ie.ie_rope(ie.Rope(D, D, 5000), Xd, posd, Y, 2 * HEADS, ws)
    want = o.rope(X, pos, o.rope_table(o.rope_frequencies(D), 5000), 2 * HEADS, D, D, False, False, o.ROW)
    assert np.array_equal(Y.exp[-LAST:].cpu().numpy(), want.exp)
    assert np.array_equal(Y.mant[-LAST:].cpu().numpy(), want.mant)
    assert not Y.mant[:LAST].any() and ws.status() == 0


def test_cache():
    announce("cache far")
    rng = np.random.default_rng(6)
    pages, page, kv, d = 8192, 256, 33, 128  # 4.4e9 bytes of keys
    assert pages * page * kv * d // 2 > 1 << 32
    k, v = (torch.empty((pages, page, kv, d // 2), dtype=torch.uint8, device="cuda") for _ in range(2))
    e, f = (torch.empty((pages, page, kv), dtype=torch.int8, device="cuda") for _ in range(2))
    cache, used = ie.Cache(k, e, v, f), [8191, 3, 8100]
    X = qkv(rng, 3 * page, kv, kv, d)
    slots = np.concatenate([np.arange(page) + p * page for p in used])
    ws = ie.Workspace("cuda")
    ie.ie_cache_store(cache, qt_to_dev(X), kv, dev_i32(slots), ws)
    small = dict(k=np.zeros((3 * page, kv, d // 2), np.uint8), v=np.zeros((3 * page, kv, d // 2), np.uint8),
                 ke=np.zeros((3 * page, kv), np.int8), ve=np.zeros((3 * page, kv), np.int8))
    o.cache_store(small, X, kv, kv, d, np.arange(3 * page))
    for name, t in (("k", k), ("ke", e), ("v", v), ("ve", f)):
        assert np.array_equal(t[used].cpu().numpy().reshape(small[name].shape), small[name]), name
    Q, O, scale = qkv(rng, 2, kv, 0, d), ie.Mat.empty(2, kv * d, ie.ROW), float(np.float32(d ** -0.5))
    table = dev_i32(np.array([used, used[::-1]]))
    ie.ie_attention_cache(ie.Attention(kv, kv, d, scale), qt_to_dev(Q), cache, table, dev_i32([700, 300]), O, ws)
    at = [np.arange(700), np.r_[2 * page:3 * page, page:page + 44]]
    assert_same(O, o.attention_cache(Q, small, at, kv, kv, d, scale), "O")
    assert ws.status() == 0
