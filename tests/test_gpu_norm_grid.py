"""Layer norm over more rows than one launch takes: 2^32 threads are refused, so the rows of workgroups of 1024 threads are split
after 2^22 - 1.  x and dy are windows into one vector, a value further from row to row; the outputs take 69 and 137 GB.  The same for the columns of dw and db, 64 to a workgroup."""
import pytest
import torch

from tests import block_ref as B
from tests import ops_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SPLIT = (1 << 22) - 1
T = SPLIT + 5
ROWS = [0, 1, SPLIT - 1, SPLIT, SPLIT + 1, T - 1]


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    return e


def windows(H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = (torch.randn(T + H - 1, generator=g, device="cuda") + 0.3).to(BF)
    return v, v.as_strided((T, H), (1, 1))


def means(v, H):
    c = torch.cat([torch.zeros(1, dtype=torch.float64, device="cuda"), torch.cumsum(v, 0)])
    return (c[H:] - c[:-H]) / H


def output(H):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 2 * T * H + (8 << 30):
        pytest.skip("the card has no %d GB free" % (2 * T * H >> 30))
    return torch.empty(T, H, dtype=BF, device="cuda")


@pytest.mark.parametrize("H", [8200, 16392])     # a row in registers, and a longer one
def test_rows(eff, H):
    v, x = windows(H, H)
    y, mean, rstd = output(H), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    y[ROWS] = float("nan")
    eff.layer_norm(x, y, mean=mean, rstd=rstd)
    for r in ROWS:
        ry, ye, rm, me, rr, re = B.norm64(x[r:r + 1].cpu(), None, None, 1e-5)
        R.assert_within(y[r:r + 1], ry, ye, "y of row %d" % r)
        R.assert_within(mean[r:r + 1], rm[:, 0], me[:, 0], "mean")
        R.assert_within(rstd[r:r + 1], rr[:, 0], re[:, 0], "rstd")
    # every row's mean; the bound is norm64's, with 2 mean |x| for the mean of the deviations' magnitudes
    D, a = B.depth(H), means(v.double().abs(), H)
    first = (D + 4) * B.U * a
    R.assert_within(mean, means(v.double(), H), (D + 6) * B.U * (2 * a + first) + 2 * B.U * (a + first), "means")
    del y
    torch.cuda.empty_cache()


def test_gradients(eff):
    H = 16392
    (v, x), (_, dy) = windows(H, 1), windows(H, 2)
    m = means(v.double(), H)
    mean, rstd = m.float(), (means(v.double() ** 2, H) - m * m + 1e-5).rsqrt().float()
    dx = output(H)
    dx[ROWS] = float("nan")
    eff.layer_norm_backward(dy, x, mean, rstd, dx=dx)
    for r in ROWS:
        rx, xe = B.norm_grad64(dy[r:r + 1].cpu(), x[r:r + 1].cpu(), None, mean[r:r + 1].cpu(), rstd[r:r + 1].cpu(), None)[:2]
        R.assert_within(dx[r:r + 1], rx, xe, "dx of row %d" % r)
    del dx
    torch.cuda.empty_cache()


def test_columns(eff):
    """dw and db of more columns than the last launch adds up at once."""
    H = 64 * SPLIT + 4099
    g = torch.Generator(device="cuda").manual_seed(3)
    x, dy = [torch.randn(1, H, generator=g, device="cuda", dtype=BF) for _ in range(2)]
    mean, rstd = torch.full((1,), 0.125, device="cuda"), torch.full((1,), 0.75, device="cuda")
    dw, db = [torch.full((H,), float("nan"), device="cuda") for _ in range(2)]
    eff.layer_norm_backward(dy, x, mean, rstd, dw=dw, db=db)
    assert torch.equal(db, dy[0].float())
    for at in range(0, H, 1 << 26):
        c = slice(at, at + (1 << 26))
        want = dy[0, c].double() * (x[0, c].double() - 0.125) * 0.75
        R.assert_within(dw[c], want, 8 * B.U * want.abs(), "dw")
    del x, dy, dw, db, want
    torch.cuda.empty_cache()
