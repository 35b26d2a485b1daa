"""Outputs of attention and of the cache over arrays that the kernels read, or over each other, are refused on the host; ones
that only touch are not (the call then gets as far as its missing workspace)."""

import pytest

from integer_only_dnn_amd import ie
from tests.test_abi_attention import BIG, OK, UNSUPPORTED, WORKSPACE, att, by, cache, fwd, mat

# 8 pages of 16 slots, 2 heads of 32: 4096 bytes of keys and of values, 256 exponents each
K, V, KE, VE = 1 << 30, 1 << 31, 3 << 31, 5 << 31


def store(c, slots=1 << 36, rows=10):
    return ie.lib().ie_cache_store(by(c), 4, by(mat(rows, 256)), slots, None, BIG, None)


@pytest.mark.parametrize("slots,want", [(K, UNSUPPORTED), (K + 4092, UNSUPPORTED), (K + 4096, WORKSPACE), (K - 36, UNSUPPORTED),
                                        (K - 40, WORKSPACE), (V + 8, UNSUPPORTED), (V + 4096, WORKSPACE), (KE + 252, UNSUPPORTED),
                                        (KE + 256, WORKSPACE), (KE - 40, WORKSPACE), (VE, UNSUPPORTED), (VE - 36, UNSUPPORTED)])
def test_slots_in_the_cache(slots, want):
    assert store(cache(), slots) == want


@pytest.mark.parametrize("arrays,want", [(dict(v=K), UNSUPPORTED), (dict(v=K + 4088), UNSUPPORTED), (dict(v=K + 4096), WORKSPACE),
                                         (dict(ve=KE), UNSUPPORTED), (dict(ve=KE + 255), UNSUPPORTED), (dict(ve=KE + 256), WORKSPACE),
                                         (dict(ke=K + 4095), UNSUPPORTED), (dict(ke=K + 4096), WORKSPACE), (dict(ke=V - 255), UNSUPPORTED),
                                         (dict(ke=V - 256), WORKSPACE), (dict(ve=K + 7), UNSUPPORTED), (dict(ve=V + 4000), UNSUPPORTED)])
def test_arrays_of_a_cache(arrays, want):
    assert store(cache(**arrays)) == want


def test_an_empty_cache_has_no_bytes():
    assert store(cache(k=0, v=0, ke=0, ve=0, pages=0)) == WORKSPACE
    assert ie.lib().ie_cache_store(by(cache()), 4, by(mat(0, 256)), K, 1, BIG, None) == OK


@pytest.mark.parametrize("at,want", [(0, UNSUPPORTED), (312, UNSUPPORTED), (316, UNSUPPORTED), (320, WORKSPACE), (-8, UNSUPPORTED),
                                     (-12, WORKSPACE)])
def test_stats_over_the_offsets(at, want):
    """10 rows of 4 heads have 320 bytes of statistics, two sequences 12 bytes of offsets."""
    assert fwd(att(n_seq=2, offsets=(1 << 40) + at), stats=1 << 40) == want
