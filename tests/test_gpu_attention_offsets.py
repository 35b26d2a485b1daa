"""Offsets that break the rules: what is undefined then, and what is not."""

import numpy as np
import pytest
import torch

import oracle as o
from integer_only_dnn_amd import ie
from tests.attention_util import SENTINEL, dev_i32, qkv, to_dev
from tests.gpu_util import announce, rand_qt

pytestmark = pytest.mark.gpu


class Guarded:
    """A device array between guard bytes."""

    def __init__(self, numel, dtype=torch.int8):
        self.buf = torch.full((numel + 8192,), SENTINEL, dtype=dtype, device="cuda")
        self.view = self.buf[4096:4096 + numel]

    def whole(self):
        return bool((self.buf[:4096] == SENTINEL).all()) and bool((self.buf[-4096:] == SENTINEL).all())


def calls(X, heads, kv, d, causal, offsets, dO):
    """Both passes between guards: (O, dQKV) on the host, after the flag and the guards are checked."""
    rows = X.mant.shape[0]
    att, ws = ie.Attention(heads, kv, d, 0.25, causal, dev_i32(offsets)), ie.Workspace("cuda")
    ws.get(max(ie.lib().ie_attention_fwd_workspace(att.desc, rows), ie.lib().ie_attention_bwd_workspace(att.desc, rows)))
    ws.buf[256:].fill_(0x5a)
    guards = [Guarded(n) for n in (rows * heads * d, rows, rows * (heads + 2 * kv) * d, rows)]
    stats = Guarded(rows * heads * 2, torch.int32)
    O = ie.Mat(guards[0].view.view(rows, -1), guards[1].view, ie.ROW)
    G = ie.Mat(guards[2].view.view(rows, -1), guards[3].view, ie.ROW)
    Xd = to_dev(X)
    ie.ie_attention_fwd(att, Xd, O, ws, stats.view)
    assert ws.status() & ie.FLAG_INDEX  # undefined rows may set the exponents' flag too
    ie.ie_attention_bwd(att, Xd, O, to_dev(dO), stats.view, G, ws)
    assert ws.status() & ie.FLAG_INDEX  # undefined rows may set the exponents' flag too
    assert all(g.whole() for g in guards) and stats.whole()
    return [(m.mant.cpu().numpy(), m.exp.cpu().numpy()) for m in (O, G)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("offsets", [[0, 1000, 500, 1000, 1100], [0, 1000, 0, 1000, 0, 1000, 1100], [1100, 0, 1100, 0], [0, 50, 40] + 80 * [60, 1100, 30]],
                         ids=["back", "over", "down", "many"])
def test_falling_offsets_write_nothing_else(offsets, causal):
    announce(f"falling offsets {offsets[:5]} {causal}")
    rng = np.random.default_rng(len(offsets))
    X = qkv(rng, 1100, 2, 1, 16)
    calls(X, 2, 1, 16, causal, offsets, rand_qt(rng, (1100, 32), o.ROW, -12, -9))


@pytest.mark.parametrize("causal", [False, True])
def test_other_sequences_are_right(causal):
    """Offsets before and past the matrix: the sequences between them are what they are without them."""
    announce(f"offsets outside {causal}")
    rng = np.random.default_rng(5)
    X, dO = qkv(rng, 700, 4, 2, 32), rand_qt(rng, (700, 128), o.ROW, -12, -9)
    for offsets, good in (([-7, 20, 300, 301, 650, 1 << 30], (20, 650)), ([0, 20, 300, 301, 650, 701], (0, 650)),
                          ([-(1 << 31), 20, 300, 301, 650, 700], (20, 700))):
        (m, e), (gm, ge) = calls(X, 4, 2, 32, causal, offsets, dO)
        inside = [t for t in offsets if good[0] <= t <= good[1]]
        want, top, total = o.attention_fwd(X, 4, 2, 32, 0.25, causal, inside)
        at = slice(*good)
        assert np.array_equal(m[at], want.mant[at]) and np.array_equal(e[at], want.exp[at])
        wantG = o.attention_bwd(X, want, dO, top, total, 4, 2, 32, 0.25, causal, inside)
        assert np.array_equal(gm[at], wantG.mant[at]) and np.array_equal(ge[at], wantG.exp[at])


@pytest.mark.parametrize("causal", [False, True])
def test_a_sequence_that_is_too_long(causal):
    """131072 tokens and more in one sequence (half as many in the gradient, where two heads share a key): those in front of it
    and behind it are right."""
    announce(f"too long {causal}")
    rng = np.random.default_rng(6)
    rows, offsets = 131300, [0, 60, 131200, 131300]
    X, dO = qkv(rng, rows, 2, 1, 16), rand_qt(rng, (rows, 32), o.ROW, -12, -9)
    (m, e), (gm, ge) = calls(X, 2, 1, 16, causal, offsets, dO)
    for a, b in ((0, 60), (131200, 131300)):
        x, dy = (o.QT(t.mant[a:b], t.exp[a:b], o.ROW) for t in (X, dO))
        want, top, total = o.attention_fwd(x, 2, 1, 16, 0.25, causal)
        assert np.array_equal(m[a:b], want.mant) and np.array_equal(e[a:b], want.exp)
        wantG = o.attention_bwd(x, want, dy, top, total, 2, 1, 16, 0.25, causal)
        assert np.array_equal(gm[a:b], wantG.mant) and np.array_equal(ge[a:b], wantG.exp)
