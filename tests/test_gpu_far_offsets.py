"""The block operators on matrices of more than 2^32 mantissas: rows on both
sides of the 2^31st and 2^32nd byte, and the last ones, against the oracle."""

import numpy as np
import pytest
import torch

import oracle as o
from integer_only_dnn_amd import ie
from tests.gpu_util import announce, qt_to_dev, rand_qt

pytestmark = pytest.mark.gpu

R = o.ROW
ROWS, COLS = 5600000, 768  # 4.3e9 mantissas
EPS = o.Scalar(85, -23)
# rows around the bytes that 31 and 32 bits end at (of mantissas, and of 16-bit values between two passes), and both ends
EDGES = [(1 << bits) // pitch for bits in (31, 32) for pitch in (COLS, 1027, 2 * 1032)]
SOME = np.unique(np.r_[0:3, [e + k for e in EDGES for k in (-2, -1, 0, 1)], ROWS - 70:ROWS])


@pytest.fixture(scope="module")
def big():
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("less than 60 GiB of device memory free")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def mat():
        m = torch.randint(-128, 128, (ROWS, COLS), generator=g, dtype=torch.int8, device="cuda")
        e = torch.randint(-14, -2, (ROWS,), generator=g, dtype=torch.int8, device="cuda")
        return ie.Mat(m, e, ie.ROW)
    yield mat(), mat(), ie.Mat.empty(ROWS, COLS, ie.ROW), ie.Workspace("cuda")
    torch.cuda.empty_cache()


def host(m):
    at = torch.from_numpy(SOME).cuda()
    return o.QT(m.mant[at].cpu().numpy(), m.exp[at].cpu().numpy(), R)


def same(got, want, what):
    g = host(got)
    assert np.array_equal(g.exp, want.exp) and np.array_equal(g.mant, want.mant), what


def test_norm(big):
    announce("far offsets norm")
    X, dY, Y, ws = big
    rng = np.random.default_rng(2)
    gam, bet = rand_qt(rng, (COLS, 1), R, -10, -5), rand_qt(rng, (COLS, 1), R, -10, -5)
    gd, bd, e = qt_to_dev(gam), qt_to_dev(bet), (EPS.mant, EPS.exp)
    Y.mant.fill_(77)
    ie.ie_layer_norm_fwd(X, gd, bd, e, Y, ws)
    same(Y, o.layer_norm_fwd(host(X), gam, bet, EPS, R), "Y")
    Y.mant.fill_(77)
    ie.ie_layer_norm_bwd(dY, X, gd, e, Y, None, None, ws)
    same(Y, o.layer_norm_bwd(host(dY), host(X), gam, EPS, R, R)[0], "dX")
    assert ws.status() == 0


def test_dropout(big):
    announce("far offsets dropout")
    X, D, Y, ws = big
    Y.mant.fill_(77)
    ie.ie_dropout(X, D, Y, 13107, 5, 6, ws)
    x, d = host(X), host(D)
    u = np.zeros((len(SOME), COLS), np.int64)
    for i, row in enumerate(SOME):
        for b in range(COLS // 8):
            w = o.philox4x32((b, int(row), 6, 0), (5, 0))
            u[i, 8 * b:8 * b + 8] = [w[k // 2] >> 16 * (k % 2) & 0xFFFF for k in range(8)]
    y = np.ldexp(x.mant * np.float64(np.float32(65536 / (65536 - 13107))), x.row_exp()[:, None])
    y = np.where(u >= 13107, y, 0.0) + np.ldexp(d.mant.astype(np.float64), d.row_exp()[:, None])
    same(Y, o.requant_f64(y, R), "dropout")
    assert ws.status() == 0


@pytest.mark.parametrize("cols", [COLS, 1027])
def test_product(big, cols):
    """Whole rows in a workgroup, and rows over several tiles (round to odd, rows off the runs of 16)."""
    announce(f"far offsets product {cols}")
    X, D, Y, ws = big
    rng = np.random.default_rng(3)
    W, b = rand_qt(rng, (cols, COLS), R), rand_qt(rng, (cols, 1), R, -12, -5)
    if cols != COLS:
        D, Y = None, ie.Mat.empty(ROWS, cols, ie.ROW)
    Y.mant.fill_(77)
    ie.ie_linear_fwd_fused(X, qt_to_dev(W), qt_to_dev(b), D, Y, ie.ACT_NONE, ws)
    same(Y, o.linear_fwd_fused(host(X), W, b, host(D) if D else None, R), f"product {cols}")
    assert ws.status() == 0


def test_bias_gradient(big):
    """The sums of all rows, by torch in parts: 64-bit sums of the mantissas at the largest exponent."""
    announce("far offsets bias gradient")
    X, _, _, ws = big
    db = ie.Mat.empty(COLS, 1, ie.ROW)
    ie.ie_linear_bwd_db(X, db, ws)
    top = int(X.exp.max())
    total = torch.zeros(COLS, dtype=torch.int64, device="cuda")
    for part in range(0, ROWS, 200000):
        m, s = X.mant[part:part + 200000].int(), (top - X.exp[part:part + 200000].int())[:, None]
        # half to even: the half, less one where the kept part is even
        half = torch.where(s > 0, (1 << s) >> 1, torch.zeros_like(s))
        total += torch.where(s > 0, (m + half - 1 + (m >> s & 1)) >> s, m).sum(dim=0)
    want = o.requant_np(total.cpu().numpy().reshape(-1, 1), np.full((COLS, 1), top), R, 8)
    assert np.array_equal(db.mant.cpu().numpy(), want.mant) and np.array_equal(db.exp.cpu().numpy(), want.exp)
    assert ws.status() == 0
