"""The attention operators as they are used together: a projection, rotary positions, attention and its gradient, back
through the projection (eager, captured and replayed, on two streams at once); a prompt that enters the cache and the
steps answered from it."""

import numpy as np
import pytest
import torch

import oracle as o
from integer_only_dnn_amd import ie
from tests.attention_util import dev_i32, qkv
from tests.gpu_util import announce, assert_same, qt_to_dev, rand_qt

pytestmark = pytest.mark.gpu

HEADS, KV, D, WIDTH = 4, 2, 32, 96
OFFSETS = [0, 40, 41, 41, 130]
ROWS = 130
SCALE = float(np.float32(D ** -0.5))
COLS = (HEADS + 2 * KV) * D


class Step:
    """One training step of an attention layer's products around the new operators."""

    def __init__(self, seed, causal=True):
        rng = np.random.default_rng(seed)
        self.causal = causal
        self.X, self.W = rand_qt(rng, (ROWS, WIDTH), o.ROW, -9, -6), rand_qt(rng, (COLS, WIDTH), o.ROW, -12, -9)
        self.dO = rand_qt(rng, (ROWS, HEADS * D), o.ROW, -20, -16)
        self.x, self.w, self.dy = (qt_to_dev(t) for t in (self.X, self.W, self.dO))
        e = lambda c: ie.Mat.empty(ROWS, c, ie.ROW)  # noqa: E731
        self.P, self.R, self.O, self.dR, self.dP, self.dX = e(COLS), e(COLS), e(HEADS * D), e(COLS), e(COLS), e(WIDTH)
        self.dW = ie.Mat.empty(COLS, WIDTH, ie.ROW)
        self.stats = torch.empty(ROWS, HEADS, 2, dtype=torch.int32, device="cuda")
        pos = np.concatenate([np.arange(b - a) for a, b in zip(OFFSETS[:-1], OFFSETS[1:])])
        self.pos_h, self.pos = pos, dev_i32(pos)
        self.rope = ie.Rope(D, D, 100)
        self.att = ie.Attention(HEADS, KV, D, SCALE, causal, dev_i32(OFFSETS))
        self.ws = ie.Workspace("cuda")
        self.ws.get(8 << 20)
        torch.cuda.synchronize()

    def run(self):
        ie.ie_linear_fwd(self.x, self.w, self.P, self.ws)
        ie.ie_rope(self.rope, self.P, self.pos, self.R, HEADS + KV, self.ws)
        ie.ie_attention_fwd(self.att, self.R, self.O, self.ws, self.stats)
        ie.ie_attention_bwd(self.att, self.R, self.O, self.dy, self.stats, self.dR, self.ws)
        ie.ie_rope(self.rope, self.dR, self.pos, self.dP, HEADS + KV, self.ws, inverse=True)
        ie.ie_linear_bwd_dx(self.dP, self.w, self.dX, self.ws)
        ie.ie_linear_bwd_dw(self.dP, self.x, self.dW, self.ws)

    def want(self):
        table = o.rope_table(o.rope_frequencies(D), 100)
        P = o.linear_fwd(self.X, self.W, o.ROW)
        R = o.rope(P, self.pos_h, table, HEADS + KV, D, D, False, False, o.ROW)
        O, m, L = o.attention_fwd(R, HEADS, KV, D, SCALE, self.causal, OFFSETS)
        dR = o.attention_bwd(R, O, self.dO, m, L, HEADS, KV, D, SCALE, self.causal, OFFSETS)
        dP = o.rope(dR, self.pos_h, table, HEADS + KV, D, D, False, True, o.ROW)
        return dict(P=P, R=R, O=O, dR=dR, dP=dP, dX=o.linear_bwd_dx(dP, self.W, o.ROW), dW=o.linear_bwd_dw(dP, self.X, o.ROW))

    def check(self, want, what):
        for k, t in want.items():
            assert_same(getattr(self, k), t, f"{what}: {k}")
        assert self.ws.status() == 0

    def spoil(self):
        for k in ("P", "R", "O", "dR", "dP", "dX", "dW"):
            getattr(self, k).mant.fill_(99)
        self.stats.fill_(-1)
        self.ws.buf[256:].fill_(0x37)


@pytest.mark.parametrize("causal", [True, False])
def test_training_step(causal):
    announce(f"attention layer step {causal}")
    s = Step(1, causal)
    want = s.want()
    for turn in range(2):
        s.spoil()
        s.run()
        s.check(want, f"turn {turn}")


def test_captured_step():
    """A captured step replayed on new inputs in the same tensors, with eager work between the replays."""
    announce("captured attention layer step")
    s, other = Step(2), Step(3)
    want, eager = s.want(), other.want()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.run()
    for turn in range(4):
        s.spoil()
        other.spoil()
        other.run()
        torch.cuda.synchronize()
        graph.replay()
        s.check(want, f"replay {turn}")
        other.check(eager, f"eager {turn}")
    # new inputs and new lengths in the tensors that the graph reads
    fresh = Step(4)
    for a, b in ((s.x, fresh.x), (s.w, fresh.w), (s.dy, fresh.dy)):
        a.mant.copy_(b.mant)
        a.exp.copy_(b.exp)
    graph.replay()
    s.check(fresh.want(), "new inputs")


def test_two_streams_at_once():
    announce("attention layer on two streams")
    sides = [Step(5), Step(6, False)]
    streams = [torch.cuda.Stream() for _ in sides]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, st in zip(sides, streams):
            with torch.cuda.stream(st):
                s.run()
    torch.cuda.synchronize()
    for k, s in enumerate(sides):
        s.check(s.want(), f"stream {k}")


def test_one_workspace_for_all_calls():
    """A workspace that another operator has just used, and the smallest one that the queries ask for."""
    announce("attention in a tight workspace")
    s = Step(7)
    want = s.want()
    by = s.att.desc
    need = max(ie.lib().ie_attention_fwd_workspace(by, ROWS), ie.lib().ie_attention_bwd_workspace(by, ROWS))
    buf = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    buf[:256] = 0
    s.ws.buf = buf[:need]
    ie.ie_rope(s.rope, qt_to_dev(want["P"]), s.pos, s.R, HEADS + KV, s.ws)
    ie.ie_attention_fwd(s.att, s.R, s.O, s.ws, s.stats)
    ie.ie_attention_bwd(s.att, s.R, s.O, s.dy, s.stats, s.dR, s.ws)
    for k in ("R", "O", "dR"):
        assert_same(getattr(s, k), want[k], k)
    assert bool((buf[need:] == 0x5a).all())


@pytest.mark.parametrize("page", [1, 16])
def test_prompt_then_steps(page):
    """Prompts of two sequences into the cache, then steps: each step's own keys are stored, then attended to."""
    announce(f"prompt and steps, pages of {page}")
    rng = np.random.default_rng(8)
    lengths, steps, per = [37, 5], 4, 64 // page
    pages = 2 * per + 1
    table = rng.permutation(pages)[:2 * per].reshape(2, per)
    slot = lambda i, j: table[i, j // page] * page + j % page  # noqa: E731
    host = dict(k=np.zeros((pages * page, KV, D // 2), np.uint8), v=np.zeros((pages * page, KV, D // 2), np.uint8),
                ke=np.full((pages * page, KV), -128, np.int8), ve=np.full((pages * page, KV), -128, np.int8))
    cache, ws, rope = ie.Cache.empty(pages, page, KV, D), ie.Workspace("cuda"), ie.Rope(D, D, 64)
    rtab = o.rope_table(o.rope_frequencies(D), 64)
    att, dtab = ie.Attention(HEADS, KV, D, SCALE), dev_i32(table)

    def turn(X, pos):
        R = ie.Mat.empty(X.mant.shape[0], COLS, ie.ROW)
        ie.ie_rope(rope, qt_to_dev(X), dev_i32(pos), R, HEADS + KV, ws)
        return R, o.rope(X, pos, rtab, HEADS + KV, D, D, False, False, o.ROW)

    X = qkv(rng, sum(lengths) + 2, HEADS, KV, D)  # two rows of padding
    at = np.concatenate([np.arange(t) for t in lengths] + [[0, 0]])
    slots = np.concatenate([slot(i, np.arange(t)) for i, t in enumerate(lengths)] + [[-1, -1]])
    R, Rh = turn(X, at)
    ie.ie_cache_store(cache, R, HEADS, dev_i32(slots), ws)
    o.cache_store(host, Rh, HEADS, KV, D, slots)
    for t in range(steps):
        X = qkv(rng, 2, HEADS, KV, D)
        pos = np.array(lengths) + t
        R, Rh = turn(X, pos)
        new = np.array([slot(i, pos[i]) for i in range(2)])
        ie.ie_cache_store(cache, R, HEADS, dev_i32(new), ws)
        o.cache_store(host, Rh, HEADS, KV, D, new)
        O = ie.Mat.empty(2, HEADS * D, ie.ROW)
        ie.ie_attention_cache(att, R, cache, dtab, dev_i32(pos + 1), O, ws)
        rows = [slot(i, np.arange(pos[i] + 1)) for i in range(2)]
        assert_same(O, o.attention_cache(Rh, host, rows, HEADS, KV, D, SCALE), f"step {t}")
    assert ws.status() == 0


def test_captured_steps_follow_their_lengths():
    """A captured decode step reads lengths and pages anew on every replay."""
    announce("captured cache step")
    rng = np.random.default_rng(9)
    page, per = 8, 100
    cache = ie.Cache(*(torch.from_numpy(a).cuda() for a in (
        rng.integers(0, 256, (per + 2, page, KV, D // 2)).astype(np.uint8), rng.integers(-5, 0, (per + 2, page, KV)).astype(np.int8),
        rng.integers(0, 256, (per + 2, page, KV, D // 2)).astype(np.uint8), rng.integers(-5, 0, (per + 2, page, KV)).astype(np.int8))))
    host = {k: t.cpu().numpy().reshape(-1, *t.shape[2:]) for k, t in (("k", cache.k), ("ke", cache.k_exp), ("v", cache.v), ("ve", cache.v_exp))}
    Q = qkv(rng, 2, HEADS, KV, D)
    q, O, ws, att = qt_to_dev(Q), ie.Mat.empty(2, HEADS * D, ie.ROW), ie.Workspace("cuda"), ie.Attention(HEADS, KV, D, SCALE)
    table, lengths = dev_i32(np.zeros((2, per))), dev_i32([1, 1])
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        ie.ie_attention_cache(att, q, cache, table, lengths, O, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        ie.ie_attention_cache(att, q, cache, table, lengths, O, ws)
    for lens in ([1, 2], [800, 0], [256, 257], [3, 799], [1, 2]):
        pages = np.stack([rng.permutation(per + 2)[:per] for _ in range(2)])
        table.copy_(dev_i32(pages))
        lengths.copy_(dev_i32(lens))
        torch.cuda.synchronize()
        graph.replay()
        slots = [pages[i, np.arange(n) // page] * page + np.arange(n) % page for i, n in enumerate(lens)]
        assert_same(O, o.attention_cache(Q, host, slots, HEADS, KV, D, SCALE), str(lens))
    assert ws.status() == 0
