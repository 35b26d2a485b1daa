"""What the attention, rotary and cache entry points refuse on the host, before anything is enqueued."""

import ctypes
import math

import pytest
import torch

from integer_only_dnn_amd import ie

by = ctypes.byref
BIG = 1 << 40
OK, NULL, SHAPE, GROUP, WORKSPACE, UNSUPPORTED, BITS = 0, 1, 2, 3, 4, 6, 8


def mat(rows, cols, mant=1 << 20, group=1, bits=0, exp=None):
    return ie.ie_mat(mant, (mant + (1 << 32)) if exp is None else exp, rows, cols, group, bits)


def att(heads=4, kv=2, d=32, causal=0, scale=0.25, n_seq=0, offsets=None):
    return ie.ie_attention_desc(heads, kv, d, causal, scale, n_seq, offsets)


def fwd(a=None, X=None, O=None, stats=None, ws=None, ws_bytes=BIG):
    """A call that gets as far as its missing workspace unless something else is wrong."""
    L = ie.lib()
    a = a if a is not None else att()
    X = X if X is not None else mat(10, 256)
    O = O if O is not None else mat(10, 128, 1 << 24)
    return L.ie_attention_fwd(by(a), by(X), by(O), stats, ws, ws_bytes, None)


def bwd(a=None, X=None, O=None, dO=None, G=None, stats=1 << 35, ws=None, ws_bytes=BIG):
    L = ie.lib()
    a = a if a is not None else att()
    X = X if X is not None else mat(10, 256)
    O = O if O is not None else mat(10, 128, 1 << 24)
    dO = dO if dO is not None else mat(10, 128, 1 << 26)
    G = G if G is not None else mat(10, 256, 1 << 28)
    return L.ie_attention_bwd(by(a), by(X), by(O), by(dO), stats, by(G), ws, ws_bytes, None)


def test_attention_forward():
    L = ie.lib()
    assert fwd() == WORKSPACE
    assert L.ie_attention_fwd(None, by(mat(10, 256)), by(mat(10, 128)), None, 1, BIG, None) == NULL
    assert L.ie_attention_fwd(by(att()), None, by(mat(10, 128)), None, 1, BIG, None) == NULL
    assert fwd(ws=1, ws_bytes=256) == WORKSPACE
    for bad in (att(heads=0), att(kv=0), att(d=0), att(heads=3), att(heads=-4), att(n_seq=-1, offsets=4), att(n_seq=2),
                att(offsets=1 << 30)):
        assert fwd(bad) == SHAPE, bad
    for bad in (att(d=129), att(scale=0.0), att(scale=-1.0), att(scale=math.inf), att(scale=math.nan), att(scale=2.0 ** 31),
                att(scale=2.0 ** -31), att(n_seq=2, offsets=(1 << 30) + 2)):
        n = (bad.heads + 2 * bad.kv_heads) * bad.head_dim
        assert fwd(bad, mat(10, n), mat(10, bad.heads * bad.head_dim, 1 << 24)) == UNSUPPORTED
    assert fwd(X=mat(10, 255)) == SHAPE and fwd(O=mat(9, 128, 1 << 24)) == SHAPE and fwd(O=mat(10, 64, 1 << 24)) == SHAPE
    assert fwd(X=mat(10, 256, group=5)) == GROUP and fwd(O=mat(10, 128, 1 << 24, bits=1)) == BITS
    assert fwd(O=mat(10, 128, 1 << 24, group=0)) == UNSUPPORTED  # one exponent a token
    assert fwd(stats=(1 << 35) + 4) == UNSUPPORTED
    assert fwd(X=mat(10, 256, mant=0, exp=5)) == NULL
    # outputs over an input, the offsets or the statistics
    assert fwd(O=mat(10, 128, (1 << 20) + 2559)) == UNSUPPORTED
    assert fwd(O=mat(10, 128, 1 << 24, exp=(1 << 20) + 5)) == UNSUPPORTED
    assert fwd(att(n_seq=1, offsets=(1 << 24) + 1276)) == UNSUPPORTED
    assert fwd(stats=(1 << 24) + 1272) == UNSUPPORTED and fwd(stats=(1 << 20) + 2552) == UNSUPPORTED
    assert fwd(stats=(1 << 20) + 2560) == WORKSPACE and fwd(O=mat(10, 128, (1 << 20) + 2560)) == WORKSPACE
    # more workgroups than a launch takes, and a single sequence that is too long
    at = dict(n_seq=4, offsets=1 << 45)
    for heads, rows, want in ((4, (1 << 26) - 4, WORKSPACE), (4, (1 << 26) - 3, UNSUPPORTED), (128, (1 << 22) - 448, WORKSPACE),
                              (128, 1 << 22, UNSUPPORTED)):
        assert fwd(att(heads, heads, 1, **at), mat(rows, 3 * heads), mat(rows, heads, 1 << 50)) == want, (heads, rows)
    assert fwd(att(n_seq=(1 << 22) - 10, offsets=1 << 45)) == WORKSPACE and fwd(att(n_seq=1 << 22, offsets=1 << 45)) == UNSUPPORTED
    assert fwd(X=mat(131071, 256), O=mat(131071, 128, 1 << 50)) == WORKSPACE
    assert fwd(X=mat(131072, 256), O=mat(131072, 128, 1 << 50)) == UNSUPPORTED
    # nothing to do
    assert fwd(X=mat(0, 256), O=mat(0, 128, 1 << 24), ws=1) == OK


def test_attention_backward():
    L = ie.lib()
    assert bwd() == WORKSPACE and bwd(ws=1, ws_bytes=256) == WORKSPACE
    assert L.ie_attention_bwd(None, by(mat(10, 256)), by(mat(10, 128)), by(mat(10, 128)), 8, by(mat(10, 256)), 1, BIG, None) == NULL
    assert bwd(stats=None) == NULL and bwd(stats=(1 << 35) + 4) == UNSUPPORTED
    assert bwd(O=mat(10, 96, 1 << 24)) == SHAPE and bwd(dO=mat(11, 128, 1 << 26)) == SHAPE and bwd(G=mat(10, 128, 1 << 28)) == SHAPE
    assert bwd(O=mat(10, 128, 1 << 24, group=0)) == UNSUPPORTED and bwd(G=mat(10, 256, 1 << 28, group=0)) == UNSUPPORTED
    assert bwd(dO=mat(10, 128, 1 << 26, group=0)) == WORKSPACE
    for m in ((1 << 20) + 1, (1 << 24) + 1, (1 << 26) - 2559, (1 << 35) + 319):
        assert bwd(G=mat(10, 256, m)) == UNSUPPORTED, m
    assert bwd(G=mat(10, 256, (1 << 35) + 320)) == WORKSPACE
    assert bwd(att(n_seq=1, offsets=1 << 28)) == UNSUPPORTED
    for rows, want in ((65535, WORKSPACE), (65536, UNSUPPORTED)):  # two query heads to a key head
        assert bwd(None, mat(rows, 256), mat(rows, 128, 1 << 50), mat(rows, 128, 1 << 52), mat(rows, 256, 1 << 54), 1 << 56) == want
    wide = att(heads=1 << 18, kv=1, d=1)
    assert bwd(wide, mat(1, (1 << 18) + 2), mat(1, 1 << 18, 1 << 30), mat(1, 1 << 18, 1 << 33), mat(1, (1 << 18) + 2, 1 << 34)) == \
        UNSUPPORTED


def freqs(base=1e4, factor=1.0, trained=0.0, low=1.0, high=4.0):
    return ie.ie_rope_freqs(base, factor, trained, low, high)


def test_rope_table():
    L = ie.lib()
    call = lambda f, rot=8, n=4, t=1 << 20: L.ie_rope_table(by(f), rot, n, t, None)  # noqa: E731
    assert L.ie_rope_table(None, 8, 4, 1 << 20, None) == NULL and call(freqs(), t=None) == NULL
    assert call(freqs(), rot=-2) == SHAPE and call(freqs(), n=-1) == SHAPE
    assert call(freqs(), rot=7) == UNSUPPORTED and call(freqs(), rot=514) == UNSUPPORTED and call(freqs(), t=(1 << 20) + 8) == UNSUPPORTED
    for bad in (freqs(base=0.0), freqs(base=math.nan), freqs(factor=0.0), freqs(factor=math.inf), freqs(trained=-1.0),
                freqs(trained=10.0, low=4.0), freqs(trained=10.0, high=math.nan)):
        assert call(bad) == UNSUPPORTED
    assert call(freqs(), rot=0, t=None) == OK and call(freqs(), n=0, t=None) == OK


def rope(X=None, Y=None, ws=None, ws_bytes=BIG, **k):
    d = dict(table=1 << 40, positions=100, pos=None, heads=4, head_dim=32, rot=32, interleaved=0, inverse=0)
    d.update(k)
    X, Y = X if X is not None else mat(10, 256), Y if Y is not None else mat(10, 256, 1 << 24)
    return ie.lib().ie_rope(by(ie.ie_rope_desc(*d.values())), by(X), by(Y), ws, ws_bytes, None)


def test_rope():
    assert rope() == WORKSPACE and rope(ws=1, ws_bytes=256) == WORKSPACE
    assert ie.lib().ie_rope(None, by(mat(1, 8)), by(mat(1, 8)), 1, BIG, None) == NULL
    assert rope(table=None) == NULL and rope(table=None, rot=0) == WORKSPACE
    assert rope(heads=9) == SHAPE and rope(heads=-1) == SHAPE and rope(rot=34) == SHAPE and rope(positions=0) == SHAPE
    assert rope(head_dim=0) == SHAPE and rope(Y=mat(10, 255, 1 << 24)) == SHAPE
    assert rope(rot=31) == UNSUPPORTED and rope(table=(1 << 40) + 8) == UNSUPPORTED and rope(pos=(1 << 41) + 2) == UNSUPPORTED
    assert rope(X=mat(1, 4096), Y=mat(1, 4096, 1 << 24), heads=1, head_dim=4096, rot=514) == UNSUPPORTED
    assert rope(Y=mat(10, 256)) == UNSUPPORTED and rope(Y=mat(10, 256, (1 << 20) + 2559)) == UNSUPPORTED
    assert rope(Y=mat(10, 256, (1 << 40) + 16)) == UNSUPPORTED and rope(pos=(1 << 24) + 4) == UNSUPPORTED


def cache(k=1 << 30, v=1 << 31, ke=3 << 31, ve=5 << 31, pages=8, page=16, kv=2, d=32):
    return ie.ie_cache(k, v, ke, ve, pages, page, kv, d)


def test_cache_store():
    L = ie.lib()

    def call(c=None, heads=4, X=None, slots=1 << 36, ws=None, ws_bytes=BIG):
        c, X = c if c is not None else cache(), X if X is not None else mat(10, 256)
        return L.ie_cache_store(by(c), heads, by(X), slots, ws, ws_bytes, None)

    assert call() == WORKSPACE and call(ws=1, ws_bytes=255) == WORKSPACE
    assert L.ie_cache_store(None, 4, by(mat(10, 256)), 4, 1, BIG, None) == NULL
    for z in ("k", "v", "ke", "ve"):
        assert call(cache(**{z: None})) == NULL
    assert call(slots=None) == NULL and call(slots=(1 << 36) + 1) == UNSUPPORTED
    for z in (dict(pages=-1), dict(page=0), dict(kv=0), dict(d=0)):
        assert call(cache(**z)) == SHAPE
    for z in (dict(page=24), dict(d=24, kv=2), dict(d=144), dict(pages=1 << 28, page=256), dict(k=(1 << 30) + 4), dict(v=(1 << 31) + 4),
              dict(kv=70000)):
        c = cache(**z)
        assert call(c, X=mat(10, (4 + 2 * c.kv_heads) * c.head_dim)) == UNSUPPORTED, z
    assert call(heads=5) == SHAPE and call(heads=-1) == SHAPE
    assert call(X=mat(10, 256, (1 << 30) + 5)) == UNSUPPORTED and call(X=mat(10, 256, (5 << 31) - 100)) == UNSUPPORTED
    assert call(X=mat(0, 256), slots=None, ws=1) == OK


def test_cache_attention():
    L = ie.lib()

    def call(a=None, Q=None, c=None, pages=1 << 36, per=4, lengths=1 << 37, O=None, ws=None, ws_bytes=BIG):
        a, c = a if a is not None else att(), c if c is not None else cache()
        Q, O = Q if Q is not None else mat(10, 256), O if O is not None else mat(10, 128, 1 << 24)
        return L.ie_attention_cache(by(a), by(Q), by(c), pages, per, lengths, by(O), ws, ws_bytes, None)

    assert call() == WORKSPACE and call(Q=mat(10, 128)) == WORKSPACE and call(ws=1, ws_bytes=256) == WORKSPACE
    assert call(pages=None) == NULL and call(lengths=None) == NULL and call(pages=None, per=0) == WORKSPACE
    assert call(Q=mat(10, 160)) == SHAPE and call(per=-1) == SHAPE and call(O=mat(9, 128, 1 << 24)) == SHAPE
    assert call(c=cache(kv=4)) == SHAPE and call(c=cache(d=16)) == SHAPE and call(att(n_seq=1, offsets=4)) == SHAPE
    assert call(O=mat(10, 128, 1 << 24, group=0)) == UNSUPPORTED and call(lengths=(1 << 37) + 2) == UNSUPPORTED
    assert call(per=(1 << 19) + 1) == UNSUPPORTED and call(att(scale=0.0)) == UNSUPPORTED
    for o in (1 << 20, 1 << 30, (1 << 31) + 2048, (3 << 31) + 100, (1 << 36) + 159, (1 << 37) + 39):
        assert call(O=mat(10, 128, o)) == UNSUPPORTED, o
    assert call(O=mat(10, 128, (1 << 37) + 40)) == WORKSPACE
    assert call(Q=mat(0, 256), O=mat(0, 128, 1 << 24), ws=1, pages=None, lengths=None) == OK
    for n, want in (((1 << 22) - 1, WORKSPACE), (1 << 22, UNSUPPORTED)):
        assert call(Q=mat(n, 128), O=mat(n, 128, 1 << 44), per=0, pages=None, lengths=1 << 50) == want
    big = mat(1 << 20, 256)
    assert call(Q=big, O=mat(1 << 20, 128, 1 << 44), per=1 << 19) == UNSUPPORTED


def test_workspace_queries():
    L = ie.lib()
    assert L.ie_attention_fwd_workspace(None, 5) == 0 and L.ie_attention_fwd_workspace(by(att()), -1) == 0
    assert L.ie_attention_bwd_workspace(by(att(d=129)), 5) == 0 and L.ie_attention_cache_workspace(by(att()), 1, -1) == 0
    assert L.ie_rope_workspace(-1, 5) == 0
    a = att()
    assert L.ie_attention_fwd_workspace(by(a), 100) >= 256 + 100 * 128 * 2 + 100 * 4 * 2
    assert L.ie_attention_bwd_workspace(by(a), 100) >= 100 * (256 * 2 + 8 * 2 + 4 * 8 + 2 + 4 * 32 + 2 * 4)
    assert L.ie_attention_cache_workspace(by(a), 3, 1000) >= 3 * 4 * (128 * 4 + 4 * 16)


class _OnGpu(torch.Tensor):
    """A host tensor that says it is on the GPU."""
    is_cuda = property(lambda self: True)


def gpu(*shape, dtype=torch.int8):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnGpu)


def test_binding():
    i32 = torch.int32
    with pytest.raises(ValueError):
        ie.Attention(4, 2, 32, 0.25, True, torch.zeros(3, dtype=i32))  # in host memory
    with pytest.raises(ValueError):
        ie.Attention(4, 2, 32, 0.25, True, gpu(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        ie.Attention(4, 2, 32, 0.25, True, gpu(1, dtype=i32))
    with pytest.raises(ValueError):
        ie.Attention(4, 2, 32, 0.25, True, gpu(6, dtype=i32)[::2])
    a, ws = ie.Attention(4, 2, 32, 0.25, True, gpu(3, dtype=i32)), ie.Workspace("cpu")
    assert (a.desc.n_seq, a.desc.causal) == (2, 1)
    X, O = ie.Mat(gpu(10, 256), gpu(10), ie.ROW), ie.Mat(gpu(10, 128), gpu(10), ie.ROW)
    for stats in (torch.zeros(10, 4, 2, dtype=i32), gpu(10, 4, 2, dtype=torch.float32), gpu(10, 4, 1, dtype=i32)):
        with pytest.raises(ValueError):
            ie.ie_attention_fwd(a, X, O, ws, stats)
        with pytest.raises(ValueError):
            ie.ie_attention_bwd(a, X, O, O, stats, X, ws)
    with pytest.raises(ValueError):
        ie.Rope(32, 32, 10, device="cpu")
    u8 = torch.uint8
    good = (gpu(2, 4, 2, 16, dtype=u8), gpu(2, 4, 2), gpu(2, 4, 2, 16, dtype=u8), gpu(2, 4, 2))
    c = ie.Cache(*good)
    assert (c.desc.pages, c.desc.page, c.desc.kv_heads, c.desc.head_dim) == (2, 4, 2, 32)
    for k, bad in ((0, gpu(2, 4, 2, 16)), (1, gpu(2, 4, 3)), (2, gpu(2, 4, 2, 8, dtype=u8)), (3, torch.zeros(2, 4, 2, dtype=torch.int8))):
        with pytest.raises(ValueError):
            ie.Cache(*[bad if i == k else t for i, t in enumerate(good)])
    with pytest.raises(ValueError):
        ie.ie_cache_store(c, X, 4, gpu(9, dtype=i32), ws)
    for pages, lengths in ((gpu(9, 2, dtype=i32), gpu(10, dtype=i32)), (gpu(10, dtype=i32), gpu(10, dtype=i32)),
                           (gpu(10, 2, dtype=i32), gpu(9, dtype=i32)), (gpu(10, 2, dtype=torch.int64), gpu(10, dtype=i32))):
        with pytest.raises(ValueError):
            ie.ie_attention_cache(a, X, c, pages, lengths, O, ws)
