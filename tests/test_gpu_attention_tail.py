"""ie_attention_fwd where most of softmax's weight lies in thousands of small weights: against the oracle bit for bit, and
against softmax in 64 bits at the longest sequence."""

import numpy as np
import pytest
import torch

import oracle as o
from integer_only_dnn_amd import ie
from tests.attention_tail import marks, sink
from tests.attention_util import assert_rows, dev_i32, filled, offsets_of, qkv, stats_of, to_dev
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu


def packed(parts):
    """Matrices of rows behind each other, one exponent a row."""
    return o.QT(np.concatenate([t.mant for t in parts]), np.concatenate([t.row_exp().astype(np.int8) for t in parts]), o.ROW)


def forward(X, heads, kv, d, scale, causal, offsets, by_stats=True):
    rows, ws = X.mant.shape[0], ie.Workspace("cuda")
    ws.get(1 << 16)
    ws.buf[256:].fill_(0x5a)
    att = ie.Attention(heads, kv, d, scale, causal, None if offsets is None else dev_i32(offsets))
    O, stats = filled(rows, heads * d), stats_of(rows, heads)
    covered = (0, rows) if offsets is None else (offsets[0], offsets[-1])
    want, m, L = o.attention_fwd(X, heads, kv, d, scale, causal, offsets)
    Xd = to_dev(X)
    for turn in range(2):  # the second one in the workspace that the first one left
        ie.ie_attention_fwd(att, Xd, O, ws, stats)
        assert_rows(O, want, covered, f"O {turn}")
        got = stats.cpu().numpy()[covered[0]:covered[1]]
        assert np.array_equal(got[..., 0], m.view(np.int32)[covered[0]:covered[1]])
        assert np.array_equal(got[..., 1], L[covered[0]:covered[1]])
    O2 = filled(rows, heads * d)
    ie.ie_attention_fwd(att, Xd, O2, ws)
    assert_rows(O2, want, covered, "O without stats")
    assert ws.status() == 0
    return want, m, L


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("n,gap,lift,mean,group", [(2033, 10.6, 0, 0.0, o.ROW), (2500, 9.4, 2, 10.0, o.ROW), (2200, 12.0, 4, 0.0, o.ROW),
                                                   (2300, 11.0, 0, 5.0, o.TENSOR)])
def test_sinks(n, gap, lift, mean, group, causal):
    announce(f"attention tail {n} {gap} {lift} {group} {causal}")
    X, scale = sink(np.random.default_rng(n), n, gap, lift=lift, mean=mean, group=group)
    m = forward(X, 1, 1, 16, scale, causal, None)[1]
    assert marks(m)[o.ATT_CHECK + (0 if causal else -1):].all()


@pytest.mark.parametrize("heads,kv,d", [(2, 1, 7), (1, 1, 40), (3, 3, 64), (2, 1, 80), (2, 2, 96), (4, 1, 128), (20, 20, 16), (16, 1, 33)])
def test_heads(heads, kv, d):
    """Few and many tiles, heads of every kernel, rows of fine weights among flat ones in each tile."""
    announce(f"attention tail heads {heads} {kv} {d}")
    X, scale = sink(np.random.default_rng(d), 2100, 10.8, heads, kv, d, lift=1, flat_rows=True)
    m = forward(X, heads, kv, d, scale, heads % 2 == 0, None)[1]
    fine = marks(m)
    assert fine[2040::2].all() and not fine[1::2].any()


@pytest.mark.parametrize("causal", [False, True])
def test_packed_with_short_ones(causal):
    """Long sequences with sinks between short ones, rows of none in front and behind; more than 64 sequences."""
    announce(f"attention tail packed {causal}")
    rng = np.random.default_rng(6)
    a, scale = sink(rng, 2200, 11.0, 2, 1, 32)
    b = sink(rng, 2077, 10.5, 2, 1, 32, lift=1)[0]
    few = [qkv(rng, t, 2, 1, 32) for t in (2, 65, 3)]
    X = packed([few[0], a, few[1], b, few[2]])
    forward(X, 2, 1, 32, scale, causal, [2, 2202, 2267, 4344])
    short = [qkv(rng, t, 2, 1, 32) for t in rng.integers(1, 30, 70)]
    X = packed([*short, a])
    forward(X, 2, 1, 32, scale, causal, offsets_of([t.mant.shape[0] for t in short] + [2200]))


def test_longest_sequence_against_softmax():
    """131071 tokens, a tail of 0.47 of the weight whose weights are a fifth of a unit each.  Tolerance: weights off by 1.2e-4
    relative twice (the exponent's resolution and cubic), half a unit of 2^-14 each, twice: 131071 * 128 / 2^14 / 61000 = 0.017
    of a mantissa's unit, half a unit of the row's rounding, and the sums of 131071 terms in float64 here."""
    announce("attention tail 131071")
    n, d = 131071, 16
    X, scale = sink(np.random.default_rng(1), n, 11.9, d=d)
    ws, O = ie.Workspace("cuda"), filled(n, d)
    ie.ie_attention_fwd(ie.Attention(1, 1, d, scale), to_dev(X), O, ws)
    assert ws.status() == 0
    rows = np.r_[0, 1, 63, 64, 65535, 131070, np.random.default_rng(2).integers(0, n, 58)]
    e = int(X.exp[0])
    x = torch.from_numpy(X.mant).cuda().double()
    t = (x[torch.from_numpy(rows).cuda(), :d] @ x[:, d:2 * d].t().contiguous()) * (2.0 ** (2 * e) * scale)
    p = torch.softmax(t, dim=1)
    want, size = (p @ x[:, 2 * d:]).cpu().numpy(), (p @ x[:, 2 * d:].abs()).cpu().numpy()
    off_sink = 1.0 - float(p[0, 0])
    assert 0.4 < off_sink < 0.55
    got = O.mant.cpu().numpy()[rows].astype(np.float64) * 2.0 ** (O.exp.cpu().numpy()[rows].astype(int) - e)[:, None]
    unit = 2.0 ** (O.exp.cpu().numpy()[rows].astype(int) - e)[:, None]
    assert np.all(np.abs(got - want) <= 2 * 1.2e-4 * size + 0.017 + 0.5 * unit)
    assert np.abs(want).max() > 0.1  # coarse weights give zeros


def test_captured_and_replayed():
    """A captured call on inputs with and without such rows, by turns: the mark of the one is not seen by the other."""
    announce("attention tail captured")
    n, d = 2100, 32
    A, scale = sink(np.random.default_rng(1), n, 11.0, d=d)
    B = qkv(np.random.default_rng(2), n, 1, 1, d)
    wants = [o.attention_fwd(t, 1, 1, d, scale, True)[0] for t in (A, B)]
    inputs, x = [to_dev(t) for t in (A, B)], to_dev(A)
    O, ws, att = filled(n, d), ie.Workspace("cuda"), ie.Attention(1, 1, d, scale, True)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        ie.ie_attention_fwd(att, x, O, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        ie.ie_attention_fwd(att, x, O, ws)
    for turn in (0, 1, 0, 0, 1):
        x.mant.copy_(inputs[turn].mant)
        x.exp.copy_(inputs[turn].exp)
        O.mant.fill_(3)
        torch.cuda.synchronize()
        graph.replay()
        assert_rows(O, wants[turn], (0, n), f"input {turn}")
    assert int(ws.buf[4:256].sum()) == 0 and ws.status() == 0


def gradient(X, heads, kv, d, scale, causal, offsets, seed=0):
    rng = np.random.default_rng(seed)
    rows, ws = X.mant.shape[0], ie.Workspace("cuda")
    want, m, L = o.attention_fwd(X, heads, kv, d, scale, causal, offsets)
    dO = o.QT(rng.integers(-128, 128, (rows, heads * d)).astype(np.int8), rng.integers(-16, -11, rows).astype(np.int8), o.ROW)
    wantG = o.attention_bwd(X, want, dO, m, L, heads, kv, d, scale, causal, offsets)
    covered = (0, rows) if offsets is None else (offsets[0], offsets[-1])
    ws.get(1 << 16)
    ws.buf[256:].fill_(0x5a)
    att, Xd, Yd = ie.Attention(heads, kv, d, scale, causal, None if offsets is None else dev_i32(offsets)), to_dev(X), to_dev(dO)
    O, stats, G = filled(rows, heads * d), stats_of(rows, heads), filled(rows, (heads + 2 * kv) * d)
    ie.ie_attention_fwd(att, Xd, O, ws, stats)
    for turn in range(2):
        ie.ie_attention_bwd(att, Xd, O, Yd, stats, G, ws)
        assert_rows(G, wantG, covered, f"dQKV {turn}")
    assert ws.status() == 0 and int(ws.buf[4:256].sum()) == 0
    return marks(m)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("n,gap,lift,group", [(2033, 10.6, 0, o.ROW), (2200, 12.0, 3, o.ROW), (2100, 11.0, 0, o.TENSOR)])
def test_gradient_of_sinks(n, gap, lift, group, causal):
    announce(f"attention tail gradient {n} {gap} {lift} {group} {causal}")
    X, scale = sink(np.random.default_rng(n), n, gap, lift=lift, mean=10.0, group=group)
    assert gradient(X, 1, 1, 16, scale, causal, None).any()


@pytest.mark.parametrize("heads,kv,d", [(2, 1, 7), (1, 1, 40), (3, 3, 64), (2, 1, 80), (2, 2, 96), (4, 1, 128), (16, 1, 33)])
def test_gradient_heads(heads, kv, d):
    announce(f"attention tail gradient heads {heads} {kv} {d}")
    X, scale = sink(np.random.default_rng(d), 2064, 10.8, heads, kv, d, lift=1, flat_rows=True)
    assert gradient(X, heads, kv, d, scale, heads % 2 == 0, None).any()


@pytest.mark.parametrize("causal", [False, True])
def test_gradient_packed(causal):
    """Sequences with and without such rows, one key head with and one without them; rows of none."""
    announce(f"attention tail gradient packed {causal}")
    rng = np.random.default_rng(6)
    a, scale = sink(rng, 2100, 11.0, 4, 2, 32)
    flat = qkv(rng, 2050, 4, 2, 32, elo=-9, ehi=-9)
    a.mant[:, 2 * 32:4 * 32] = flat.mant[:1, 2 * 32:4 * 32] // 16  # the second key head's queries: all scores alike
    few = [qkv(rng, t, 4, 2, 32) for t in (2, 65, 3)]
    X = packed([few[0], a, few[1], flat, few[2]])
    fine = gradient(X, 4, 2, 32, scale, causal, [2, 2102, 2167, 4217])
    assert fine[2034:2102, :2].all() and not fine[:, 2:].any() and not fine[2102:].any()
