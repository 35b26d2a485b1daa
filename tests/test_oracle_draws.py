"""The oracle's draws of a whole matrix against its generator block by block,
which tests/test_oracle_block.py pins to published values."""

import numpy as np
import pytest

import oracle as o


@pytest.mark.parametrize("shape", [(1, 1), (3, 8), (5, 41), (0, 4), (4, 0), (2, 4100)])
@pytest.mark.parametrize("seed,step", [(0, 0), ((1 << 64) - 1, (1 << 64) - 1), (0xFEDCBA9876543210, 1 << 32), (1 << 32, 5)])
def test_draws_are_the_generators(shape, seed, step):
    rows, cols = shape
    got = o.dropout_draws(rows, cols, seed, step)
    assert got.shape == shape and got.dtype == np.int64
    for i in range(rows):
        for b in {0, 1, (cols - 1) // 8} if cols > 100 else range((cols + 7) // 8):
            w = o.philox4x32((b, i, step & 0xFFFFFFFF, step >> 32), (seed & 0xFFFFFFFF, seed >> 32))
            want = [w[k // 2] >> 16 * (k % 2) & 0xFFFF for k in range(min(8, cols - 8 * b))]
            assert got[i, 8 * b:8 * b + 8].tolist() == want
