"""Attention at the ends of its range: thousands of sequences, the longest one with the largest sums, long packed batches, and
a captured call whose offsets change."""

import numpy as np
import pytest
import torch

import oracle as o
from integer_only_dnn_amd import ie
from tests.attention_tail import marks
from tests.attention_util import assert_rows, dev_i32, filled, offsets_of, qkv, stats_of, to_dev
from tests.gpu_util import announce, rand_qt
from tests.test_gpu_attention import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,causal", [(4200, True), (5000, False)])
def test_thousands_of_sequences(n, causal):
    """The search for a tile's sequence takes three turns past 4096."""
    announce(f"attention {n} sequences {causal}")
    rng = np.random.default_rng(n)
    lengths = rng.integers(0, 4, n)
    lengths[rng.integers(0, n, 3)] = 70
    rows = int(lengths.sum()) + 4
    X = qkv(rng, rows, 1, 1, 16)
    run(X, 1, 1, 16, causal, offsets_of(lengths, 1), dO=rand_qt(rng, (rows, 16), o.ROW, -12, -9))


@pytest.mark.parametrize("causal", [False, True])
def test_long_packed_batch(causal):
    """Ordinary inputs past the length from which weights are checked: no row's are fine."""
    announce(f"attention long packed {causal}")
    rng = np.random.default_rng(7)
    rows, at = 5200, [3, 2600, 2601, 4900, 5190]
    X = qkv(rng, rows, 2, 1, 32, elo=-7, ehi=-6)
    run(X, 2, 1, 32, causal, at, dO=rand_qt(rng, (rows, 64), o.ROW, -12, -9))
    assert not marks(o.attention_fwd(X, 2, 1, 32, float(np.float32(32 ** -0.5)), causal, at)[1]).any()


@pytest.mark.parametrize("n", [131071, 66060])
def test_largest_sums(n):
    """One sequence of equal tokens, all mantissas -128: every weight is 32512, digits 127 and 0, times -128; sums of 2^31 less
    2^16 at 131071.  By formula, as an n x n oracle does not fit."""
    announce(f"attention largest sums {n}")
    d, e, ed = 16, 3, -5
    X = ie.Mat(torch.full((n, 3 * d), -128, dtype=torch.int8, device="cuda"), torch.tensor([e], dtype=torch.int8, device="cuda"), ie.TENSOR)
    dO = ie.Mat(torch.full((n, d), -128, dtype=torch.int8, device="cuda"), torch.tensor([ed], dtype=torch.int8, device="cuda"), ie.TENSOR)
    ws, O, stats, G = ie.Workspace("cuda"), filled(n, d), stats_of(n, 1), filled(n, 3 * d)
    att = ie.Attention(1, 1, d, 0.25)
    ie.ie_attention_fwd(att, X, O, ws, stats)
    assert bool((O.mant == -64).all()) and bool((O.exp == e + 1).all())
    got = stats.cpu().numpy()[:, 0]
    assert np.all(got[:, 1].view(np.uint32) == n * 32512) and np.all(got[:, 0].view(np.float32) == 16 * 128 * 128 * 2.0 ** e)
    ie.ie_attention_bwd(att, X, O, dO, stats, G, ws)
    # u = 0 for every pair, so dQ and dK are zeros; dV = sum R(w a 2^-kappa) dO, one exponent of dO for all tokens
    a = np.float32(1.0 / (n * 32512))
    kappa = int(np.frexp(a)[1])
    unit = np.rint(float(np.float32(32512) * a) * 2.0 ** -kappa)
    assert unit > 32000 or n == 131071
    want = o.requant_f64(np.full((1, d), -128.0 * n * unit * 2.0 ** (kappa + ed)), o.ROW)
    assert not G.mant[:, :2 * d].any() and bool((G.mant[:, 2 * d:] == int(want.mant[0, 0])).all())
    assert bool((G.exp == int(want.exp[0])).all()) and ws.status() == 0


def test_captured_call_follows_its_offsets():
    """A captured step reads the offsets anew on every replay: other lengths, numbers of tiles and empty sequences."""
    announce("attention captured offsets")
    rng = np.random.default_rng(9)
    rows, heads, kv, d = 2300, 2, 1, 32
    X, dO = qkv(rng, rows, heads, kv, d), rand_qt(rng, (rows, heads * d), o.ROW, -12, -9)
    x, dy, at = to_dev(X), to_dev(dO), dev_i32([0, 1, 2, 3, 4])
    att, ws, scale = None, ie.Workspace("cuda"), float(np.float32(d ** -0.5))
    att = ie.Attention(heads, kv, d, scale, True, at)
    O, stats, G = filled(rows, heads * d), stats_of(rows, heads), filled(rows, (heads + 2 * kv) * d)

    def step():
        ie.ie_attention_fwd(att, x, O, ws, stats)
        ie.ie_attention_bwd(att, x, O, dy, stats, G, ws)

    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for offsets in ([0, 700, 700, 1500, 2300], [5, 6, 7, 8, 2290], [0, 0, 0, 0, 0], [100, 2200, 2250, 2250, 2251], [0, 700, 700, 1500, 2300]):
        at.copy_(dev_i32(offsets))
        for m in (O, G):
            m.mant.fill_(77)
            m.exp.fill_(77)
        torch.cuda.synchronize()
        graph.replay()
        want, top, total = o.attention_fwd(X, heads, kv, d, scale, True, offsets)
        covered = (offsets[0], offsets[-1])
        assert_rows(O, want, covered, f"O {offsets}")
        assert_rows(G, o.attention_bwd(X, want, dO, top, total, heads, kv, d, scale, True, offsets), covered, f"dQKV {offsets}")
    assert ws.status() == 0
