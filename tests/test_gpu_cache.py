"""ie_cache_store and ie_attention_cache against the oracle, bit for bit."""

import numpy as np
import pytest
import torch

import oracle as o
from integer_only_dnn_amd import ie
from tests.attention_util import dev_i32, filled, qkv, shifted
from tests.gpu_util import announce, assert_same, from_dev, qt_to_dev, rand_qt

pytestmark = pytest.mark.gpu


def new_cache(rng, pages, page, kv, d, elo=-5, ehi=0):
    host = dict(k=rng.integers(0, 256, (pages * page, kv, d // 2)).astype(np.uint8),
                v=rng.integers(0, 256, (pages * page, kv, d // 2)).astype(np.uint8),
                ke=rng.integers(elo, ehi + 1, (pages * page, kv)).astype(np.int8),
                ve=rng.integers(elo, ehi + 1, (pages * page, kv)).astype(np.int8))
    dev = {k: torch.from_numpy(v.reshape(pages, page, *v.shape[1:]).copy()).cuda() for k, v in host.items()}
    return host, ie.Cache(dev["k"], dev["ke"], dev["v"], dev["ve"])


def assert_cache(cache, host):
    torch.cuda.synchronize()
    for name, t in (("k", cache.k), ("ke", cache.k_exp), ("v", cache.v), ("ve", cache.v_exp)):
        got = t.cpu().numpy().reshape(host[name].shape)
        assert np.array_equal(got, host[name]), name


@pytest.mark.parametrize("group", [o.ROW, o.TENSOR])
@pytest.mark.parametrize("rows,heads,kv,d,page", [(1, 1, 1, 16, 1), (7, 4, 2, 32, 4), (33, 2, 2, 48, 16), (130, 8, 8, 64, 64),
                                                  (50, 0, 1, 80, 8), (20, 6, 3, 96, 2), (100, 12, 3, 112, 128), (40, 32, 8, 128, 16)])
def test_store(rows, heads, kv, d, page, group):
    announce(f"store {rows} {heads} {kv} {d} {page}")
    rng = np.random.default_rng(rows + d)
    pages = rows // page + 2
    host, cache = new_cache(rng, pages, page, kv, d)
    X = qkv(rng, rows, heads, kv, d, group, -128, 100)
    X.mant[rows // 2] = 0
    slots = rng.permutation(pages * page)[:rows]
    slots[rows // 3::5] = -1 - rng.integers(0, 9, len(slots[rows // 3::5]))
    ws = ie.Workspace("cuda")
    ie.ie_cache_store(cache, shifted(X, 3) if rows == 33 else qt_to_dev(X), heads, dev_i32(slots), ws)
    o.cache_store(host, X, heads, kv, d, slots)
    assert_cache(cache, host)
    assert ws.status() == 0


def test_slots_outside():
    announce("store outside")
    rng = np.random.default_rng(1)
    host, cache = new_cache(rng, 3, 8, 2, 32)
    X, ws = qkv(rng, 5, 2, 2, 32), ie.Workspace("cuda")
    slots = [3, 24, -1, 1 << 30, 23]
    ie.ie_cache_store(cache, qt_to_dev(X), 2, dev_i32(slots), ws)
    assert ws.status() == ie.FLAG_INDEX
    o.cache_store(host, X, 2, 2, 32, slots)
    assert_cache(cache, host)


def attend(rng, lengths, heads, kv, d, page, group=o.ROW, whole=True, bits=8, exps=(-5, 0), scale=None, spare=2, by=0):
    n, per = len(lengths), max(1, max(-(-t // page) for t in lengths)) + spare
    pages = sum(-(-t // page) for t in lengths) + 3
    host, cache = new_cache(rng, pages, page, kv, d, *exps)
    Q = qkv(rng, n, heads, kv if whole else 0, d, group)
    order, table, at, slots = rng.permutation(pages), np.full((n, per), -1), 0, []
    table[:] = rng.integers(-9, 1 << 20, table.shape)  # what lies behind a sequence's pages is not read
    for i, t in enumerate(lengths):
        k = -(-t // page)
        table[i, :k] = order[at:at + k]
        at += k
        j = np.arange(t)
        slots.append(table[i, j // page] * page + j % page)
    scale = float(np.float32(d ** -0.5)) if scale is None else scale
    ws, O = ie.Workspace("cuda"), filled(n, heads * d, bits, by)
    ws.get(1 << 16)
    ws.buf[256:].fill_(0x5a)
    att = ie.Attention(heads, kv, d, scale)
    for _ in range(2):
        ie.ie_attention_cache(att, shifted(Q, by) if by else qt_to_dev(Q), cache, dev_i32(table), dev_i32(lengths), O, ws)
        assert_same(O, o.attention_cache(Q, host, slots, heads, kv, d, scale, bits), "O")
    assert ws.status() == 0


@pytest.mark.parametrize("page", [1, 16, 256, 1024])
@pytest.mark.parametrize("lengths", [[1], [0], [255, 256, 257], [15, 0, 64, 1, 700, 33], [2100]], ids=lambda v: "+".join(map(str, v)))
def test_lengths(lengths, page):
    announce(f"cache attention {lengths} {page}")
    rng = np.random.default_rng(sum(lengths) + page)
    attend(rng, lengths, 4, 2, 32, page)


@pytest.mark.parametrize("heads,kv,d", [(1, 1, 16), (2, 2, 32), (16, 1, 48), (17, 1, 64), (40, 2, 64), (6, 3, 80), (12, 12, 96),
                                        (8, 2, 112), (32, 8, 128), (33, 33, 16), (5, 1, 64), (16, 2, 128), (14, 2, 96), (9, 1, 128),
                                        (3, 1, 48)])
@pytest.mark.parametrize("group", [o.ROW, o.TENSOR])
def test_heads(heads, kv, d, group):
    announce(f"cache attention heads {heads} {kv} {d}")
    rng = np.random.default_rng(heads + d)
    attend(rng, [300, 5, 513], heads, kv, d, 16, group, whole=heads % 2 == 0)


@pytest.mark.parametrize("exps", [(-128, 16), (-60, -40), (10, 16), (-3, -3)])
@pytest.mark.parametrize("scale", [2.0 ** -30, 1.0, 1000.0])
def test_exponents(exps, scale):
    announce(f"cache attention exponents {exps} {scale}")
    rng = np.random.default_rng(exps[1] + 99)
    attend(rng, [300, 40], 4, 2, 64, 32, exps=exps, scale=scale)


@pytest.mark.parametrize("bits,by", [(2, 0), (5, 1), (8, 4), (8, 8)])
def test_widths_and_alignment(bits, by):
    announce(f"cache attention {bits} bits, {by} off")
    attend(np.random.default_rng(bits), [77, 290], 4, 1, 64, 16, bits=bits, by=by)


@pytest.mark.parametrize("page,spare", [(8, 0), (256, 9)])
def test_many_sequences(page, spare):
    """More sequences than a workgroup scans at once, short ones and empty ones among them; tables of one and of ten blocks."""
    announce(f"cache attention many {page}")
    rng = np.random.default_rng(21)
    attend(rng, list(rng.integers(0, 40, 600)), 2, 1, 16, page, spare=spare)


@pytest.mark.parametrize("blocks", [1, 2, 4, 8, 9])
@pytest.mark.parametrize("heads,kv,d", [(8, 8, 64), (32, 4, 128), (64, 2, 16), (255, 51, 16), (257, 1, 16), (20, 4, 48)])
def test_few_blocks(heads, kv, d, blocks):
    """Tables of up to eight blocks, with the last one full, begun and empty."""
    announce(f"cache attention {blocks} blocks {heads} {kv} {d}")
    rng = np.random.default_rng(heads + blocks)
    attend(rng, [256 * blocks, 256 * blocks - 255, 256 * (blocks - 1), 1, 0], heads, kv, d, 256, spare=0)


def test_pages_and_lengths_outside():
    """Pages outside the cache leave their keys out, lengths outside the table are cut; both set the flag."""
    announce("cache attention outside")
    rng = np.random.default_rng(2)
    host, cache = new_cache(rng, 6, 16, 2, 32)
    Q, ws, O = qkv(rng, 3, 4, 2, 32), ie.Workspace("cuda"), filled(3, 128)
    att = ie.Attention(4, 2, 32, 0.25)
    table = np.array([[0, 6, 2], [-1, -1, -1], [3, 4, 5]])
    ie.ie_attention_cache(att, qt_to_dev(Q), cache, dev_i32(table), dev_i32([48, 20, 30]), O, ws)
    assert ws.status() == ie.FLAG_INDEX
    j = np.arange(48)
    slots = [np.where(j // 16 == 1, -1, table[0, j // 16] * 16 + j % 16), np.full(20, -1), table[2, j[:30] // 16] * 16 + j[:30] % 16]
    assert_same(O, o.attention_cache(Q, host, slots, 4, 2, 32, 0.25), "left out")
    table[0] = [0, 1, 2]
    table[1] = [1, 2, 0]
    ie.ie_attention_cache(att, qt_to_dev(Q), cache, dev_i32(table), dev_i32([1 << 30, -7, 30]), O, ws)
    assert ws.status() == ie.FLAG_INDEX
    slots = [table[0, j // 16] * 16 + j % 16, [], table[2, j[:30] // 16] * 16 + j[:30] % 16]
    assert_same(O, o.attention_cache(Q, host, slots, 4, 2, 32, 0.25), "cut")


def test_no_pages():
    """A table without columns: every sequence is empty, and a length above zero is told."""
    announce("cache attention without pages")
    rng = np.random.default_rng(6)
    _, cache = new_cache(rng, 2, 16, 2, 32)
    Q, ws, att = qkv(rng, 3, 4, 2, 32), ie.Workspace("cuda"), ie.Attention(4, 2, 32, 0.25)
    for lengths, flag in (([0, 0, 0], 0), ([0, 1, 0], ie.FLAG_INDEX)):
        O = filled(3, 128)
        ie.ie_attention_cache(att, qt_to_dev(Q), cache, torch.zeros((3, 0), dtype=torch.int32, device="cuda"), dev_i32(lengths), O, ws)
        assert ws.status() == flag
        assert not O.mant.any() and bool((O.exp == -128).all())


def test_shared_pages():
    """Two sequences over the same pages, and one page twice in a sequence."""
    announce("cache attention shared pages")
    rng = np.random.default_rng(3)
    host, cache = new_cache(rng, 4, 16, 1, 16)
    Q, ws, O = qkv(rng, 2, 2, 1, 16), ie.Workspace("cuda"), filled(2, 32)
    table = np.array([[1, 3, 1], [1, 3, 0]])
    ie.ie_attention_cache(ie.Attention(2, 1, 16, 0.25), qt_to_dev(Q), cache, dev_i32(table), dev_i32([48, 40]), O, ws)
    j = np.arange(48)
    slots = [table[0, j // 16] * 16 + j % 16, table[1, j[:40] // 16] * 16 + j[:40] % 16]
    assert_same(O, o.attention_cache(Q, host, slots, 2, 1, 16, 0.25), "shared")
    assert ws.status() == 0
