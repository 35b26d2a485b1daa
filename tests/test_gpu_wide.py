"""Bias gradients of rows so wide that the blocks which close the sums take
turns (2^20 columns and more), and so many that one block for each 16 of them
would be more threads than a launch has (2^26 columns)."""

import pytest
import torch

from integer_only_dnn_amd import ie
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [(1 << 20) - 1, (1 << 20) + 1, (1 << 21) + 37, (1 << 26) + 19])
@pytest.mark.parametrize("rows", [1, 3])
def test_bias_gradient_of_wide_rows(rows, cols):
    """Three mantissas of at most 42 add up to one of at most 126: the sum is exact and, with one
    exponent, the result itself; with an exponent per channel it is the sum, shifted up to fill 7 bits."""
    announce(f"wide db {rows} x {cols}")
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + cols)
    m = torch.randint(-42, 43, (rows, cols), generator=g, dtype=torch.int8, device="cuda")
    m[:, cols - 1] = 42
    m[:, 0] = 0
    if rows == 1:
        m[0, cols // 2] = 127
    want = m.sum(dim=0, dtype=torch.int32)
    assert 64 <= int(want.abs().max()) <= 127
    dY = ie.Mat(m, torch.full((rows,), -9, dtype=torch.int8, device="cuda"), ie.ROW)
    ws = ie.Workspace("cuda")
    for shape in ((cols, 1), (1, cols)):
        one = ie.Mat.empty(*shape, ie.TENSOR)
        ie.ie_linear_bwd_db(dY, one, ws)
        assert torch.equal(one.mant.view(-1).int(), want) and int(one.exp[0]) == -9
    per = ie.Mat.empty(cols, 1, ie.ROW)
    ie.ie_linear_bwd_db(dY, per, ws)
    got, e = per.mant.view(-1).int(), per.exp.int()
    zero = want == 0
    assert bool((got[zero] == 0).all()) and bool((e[zero] == -128).all())
    up = -9 - e[~zero]
    assert bool(((up >= 0) & (up <= 6)).all()) and torch.equal(got[~zero], want[~zero] << up)
    assert bool((got[~zero].abs() >= 64).all())
    assert ws.status() == 0
