"""Attention and the cache at the ends of the exponents' range, against the oracle bit for bit, and the flags they set."""

import numpy as np
import pytest
import torch

import oracle as o
from integer_only_dnn_amd import ie
from tests.attention_tail import sink
from tests.attention_util import dev_i32, filled, qkv
from tests.gpu_util import announce, assert_same, qt_to_dev, rand_qt
from tests.test_gpu_attention import run
from tests.test_gpu_cache import attend, new_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("exps", [(12, 21), (17, 21), (-10, 21)])
@pytest.mark.parametrize("scale", [2.0 ** -30, 2.0 ** -8, 1.0])
def test_large_exponents_of_a_cache(exps, scale):
    announce(f"cache exponents {exps} {scale}")
    rng = np.random.default_rng(exps[0] + 30)
    attend(rng, [300, 40, 2600], 4, 2, 64, 32, exps=exps, scale=scale)


def test_stored_rows_of_large_exponents():
    """Rows of exponents 12 to 16, which no flag is set for, stored and attended to."""
    announce("cache of large rows")
    rng = np.random.default_rng(2)
    host, cache = new_cache(rng, 4, 16, 2, 32)
    X = qkv(rng, 64, 4, 2, 32, elo=12, ehi=16)
    X.mant[:, 128:] = rng.choice([-128, 127, 100, -90, 1], X.mant[:, 128:].shape)
    ws, O = ie.Workspace("cuda"), filled(2, 128)
    slots = rng.permutation(64)
    ie.ie_cache_store(cache, qt_to_dev(X), 4, dev_i32(slots), ws)
    o.cache_store(host, X, 4, 2, 32, slots)
    assert host["ve"].max() == 21
    Q = qkv(rng, 2, 4, 0, 32, elo=-30, ehi=-25)
    ie.ie_attention_cache(ie.Attention(4, 2, 32, 0.25), qt_to_dev(Q), cache, dev_i32([[0, 1, 2, 3], [3, 1, 0, 2]]), dev_i32([64, 50]), O, ws)
    at = np.arange(64)
    table = np.array([[0, 1, 2, 3], [3, 1, 0, 2]])
    assert_same(O, o.attention_cache(Q, host, [table[0, at // 16] * 16 + at % 16, (table[1, at // 16] * 16 + at % 16)[:50]], 4, 2, 32, 0.25), "O")
    assert ws.status() == 0


@pytest.mark.parametrize("which", ["ke", "ve"])
def test_larger_ones_are_flagged(which):
    announce(f"cache flag {which}")
    rng = np.random.default_rng(3)
    host, cache = new_cache(rng, 2, 16, 1, 16)
    (cache.k_exp if which == "ke" else cache.v_exp)[1, 3, 0] = 22
    host[which][19] = 22
    Q, ws, att = qkv(rng, 1, 1, 0, 16, elo=-30, ehi=-30), ie.Workspace("cuda"), ie.Attention(1, 1, 16, 0.25)
    for length, flag in ((19, 0), (20, ie.FLAG_EXP_RANGE)):
        O = filled(1, 16)
        ie.ie_attention_cache(att, qt_to_dev(Q), cache, dev_i32([[0, 1]]), dev_i32([length]), O, ws)
        assert_same(O, o.attention_cache(Q, host, [np.arange(length)], 1, 1, 16, 0.25), "O")
        assert ws.status() == flag


@pytest.mark.parametrize("bits", [2, 3, 8])
@pytest.mark.parametrize("exps", [(16, 16), (-48, -48), (10, 16)])
def test_gradient_from_narrow_results(bits, exps):
    """O's exponents lie above 16 where its mantissas have few bits, and below -48 where small values cancel."""
    announce(f"gradient, O of {bits} bits, exponents {exps}")
    rng = np.random.default_rng(bits)
    X = qkv(rng, 70, 2, 1, 32, o.ROW, *exps)
    X.mant[:, 96:] = np.clip(X.mant[:, 96:], -2, 2) if exps[0] < 0 else np.abs(X.mant[:, 96:] // 2) + 64
    run(X, 2, 1, 32, True, None, scale=2.0 ** (-30 if exps[0] > 0 else 30), bits=bits, dO=rand_qt(rng, (70, 64), o.ROW, -20, -14))


@pytest.mark.parametrize("exps", [(-60, -50), (-126, -100), (-128, 16), (-126, -126), (-120, -30)])
@pytest.mark.parametrize("group", [o.ROW, o.TENSOR])
@pytest.mark.parametrize("scale", [2.0 ** -30, 1.0, 2.0 ** 30])
def test_small_rows(exps, group, scale):
    """Forward and gradient, short sequences and longer ones, heads of every kernel; gradients of far exponents."""
    announce(f"attention exponents {exps} {group} {scale}")
    rng = np.random.default_rng(-exps[0] + exps[1])
    for causal, rows, d in ((False, 50, 16), (True, 300, 64), (False, 290, 128)):
        X = qkv(rng, rows, 2, 1, d, group, *exps, flat=True)
        run(X, 2, 1, d, causal, [0, 1, rows], scale=scale, dO=rand_qt(rng, (rows, 2 * d), o.ROW, -128, 20))


@pytest.mark.parametrize("exps", [(-128, -100), (-128, 21), (-70, -49), (-126, -126)])
@pytest.mark.parametrize("scale", [2.0 ** -30, 1.0, 2.0 ** 30])
def test_small_exponents_of_a_cache(exps, scale):
    announce(f"cache exponents {exps} {scale}")
    attend(np.random.default_rng(exps[1] + 130), [300, 40, 2600], 4, 2, 64, 32, exps=exps, scale=scale)


def test_fine_weights_of_small_rows():
    announce("attention tail of small rows")
    X, scale = sink(np.random.default_rng(5), 2100, 10.8, lift=2)
    X.exp[:] -= 12
    run(X, 1, 1, 16, True, None, scale=scale * 2.0 ** 24, dO=rand_qt(np.random.default_rng(6), (2100, 16), o.ROW, -20, -14))
    Y = o.QT(X.mant, (X.exp.astype(int) - 100).astype(np.int8), o.ROW)  # all weights alike: every sum is large, none is fine
    run(Y, 1, 1, 16, True, None, scale=scale, dO=rand_qt(np.random.default_rng(6), (2100, 16), o.ROW, -20, -14))
