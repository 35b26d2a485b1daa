"""The README's examples of attention run as they are written."""

import os
import re

import numpy as np
import pytest
import torch

import oracle as o
from integer_only_dnn_amd import ie
from tests.attention_util import dev_i32, qkv
from tests.gpu_util import announce, assert_same, qt_to_dev, rand_qt

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_examples():
    announce("README examples")
    blocks = re.findall(r"```python\n(.*?)```", open(README).read(), re.S)
    assert len(blocks) == 2
    rng = np.random.default_rng(1)
    heads, kv_heads, head_dim, scale, positions, rows, n = 4, 2, 32, 0.25, 64, 40, 3
    X, dY = qkv(rng, rows, heads, kv_heads, head_dim), rand_qt(rng, (rows, heads * head_dim), o.ROW, -12, -9)
    at = [0, 15, 16, 40]
    place = np.concatenate([np.arange(b - a) for a, b in zip(at[:-1], at[1:])])
    e = lambda r, c: ie.Mat.empty(r, c, ie.ROW)  # noqa: E731
    width = (heads + 2 * kv_heads) * head_dim
    names = dict(ie=ie, heads=heads, kv_heads=kv_heads, head_dim=head_dim, scale=scale, positions=positions, offsets=dev_i32(at),
                 pos=dev_i32(place), QKV=qt_to_dev(X), QKVr=e(rows, width), O=e(rows, heads * head_dim), dO=qt_to_dev(dY),
                 stats=torch.empty(rows, heads, 2, dtype=torch.int32, device="cuda"), dQKVr=e(rows, width), dQKV=e(rows, width),
                 ws=ie.Workspace("cuda"))
    exec(blocks[0], names)
    table = o.rope_table(o.rope_frequencies(head_dim), positions)
    R = o.rope(X, place, table, heads + kv_heads, head_dim, head_dim, False, False, o.ROW)
    O, m, L = o.attention_fwd(R, heads, kv_heads, head_dim, scale, True, at)
    G = o.attention_bwd(R, O, dY, m, L, heads, kv_heads, head_dim, scale, True, at)
    assert_same(names["O"], O, "O")
    assert_same(names["dQKV"], o.rope(G, place, table, heads + kv_heads, head_dim, head_dim, False, True, o.ROW), "dQKV")
    # a server's step: three sequences' first tokens, in the names that the step in front has left
    Y = qkv(rng, n, heads, kv_heads, head_dim)
    slots = [5, 16, 40]
    names.update(QKVr=qt_to_dev(Y), slots=dev_i32(slots), pages=4, page=16, table=dev_i32([[0, 1], [1, 0], [2, 3]]),
                 lengths=dev_i32([6, 1, 9]), O=e(n, heads * head_dim))
    exec(blocks[1], names)
    host = {k: np.zeros((64, kv_heads, head_dim // 2), np.uint8) for k in ("k", "v")}
    host.update({k: np.full((64, kv_heads), -128, np.int8) for k in ("ke", "ve")})
    o.cache_store(host, Y, heads, kv_heads, head_dim, slots)
    want = o.attention_cache(Y, host, [np.arange(6), np.array([16]), np.arange(32, 41)], heads, kv_heads, head_dim, scale)
    assert_same(names["O"], want, "step")
    assert names["ws"].status() == 0
