"""Joining the blocks of a cache: exact sums, whatever their size and order."""

import numpy as np

import oracle as o


def test_sums_of_the_largest_caches_are_exact():
    """2^23 positions, all weights near one, values of 7 and -8: sums of up to 2^55.9, where float64 rounds."""
    rng = np.random.default_rng(1)
    blocks, d = 1 << 15, 4
    lb = rng.integers(250 * 32512, 256 * 32512 + 1, blocks)
    nb = rng.choice([7, -8], (blocks, 1)) * lb[:, None] - rng.integers(0, 9, (blocks, d))
    nb[:, 1], nb[:, 2] = np.abs(nb[:, 1]), -np.abs(nb[:, 2])
    m = -rng.integers(0, 300, blocks) * 2.0 ** -12
    total, num, top = o.cache_join([(m[b], lb[b], 0, nb[b].astype(np.float64)) for b in range(blocks)], np.float64(1.0))
    w = [int(x) for x in np.rint(o.softmax_weight(o.ie_oracle._f32(m - m.max()), np.float64(1.0)))]
    assert top == 0 and int(total) == sum(a * int(b) for a, b in zip(w, lb))
    want = [sum(a * int(b) for a, b in zip(w, nb[:, k])) for k in range(d)]
    assert max(abs(x) for x in want) > 1 << 55
    assert [int(x) for x in num] == want
    # in float64, as rounded sums, they differ from it and from one order to another
    floats = np.cumsum(np.array(w, float)[:, None] * nb, axis=0)[-1]
    assert any(int(f) != x for f, x in zip(floats, want))
