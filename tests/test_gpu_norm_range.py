"""Layer norm of rows whose squared deviations, or whose sum, are beyond fp32, although every value and every result is within it."""
import pytest
import torch

from tests import block_ref as B
from tests import ops_ref as R
from tests.test_gpu_norm import check, rows, weights

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
LENGTHS = [1, 2, 40, 257, 512, 1000, 2048, 4096, 8192, 8200, 16400, 40001]   # every shape of the row kernels


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    return e


@pytest.mark.parametrize("H", LENGTHS)
@pytest.mark.parametrize("dt", [BF, F32])
def test_squares_beyond_fp32(eff, H, dt):
    """Spreads about 2^62, where the sum of squares begins to overflow, and far above it; the last ones' sums overflow too."""
    for scale in (2.0 ** 62, 1e25, 3e35, 4e37):
        check(eff, rows(5, H, dt, H, 0.3) * scale, weights(H, F32, H), weights(H, F32, H + 1, 1.0))


@pytest.mark.parametrize("H", LENGTHS)
@pytest.mark.parametrize("dt", [BF, F32])
def test_squares_below_fp32(eff, H, dt):
    """eps 0 or next to nothing: the row's own spread decides, however small it is."""
    for scale, eps in ((1e-18, 0.0), (1e-25, 0.0), (1e-18, 1e-37), (1e-20, 1e-40), (1e-30, 0.0)):
        x = rows(5, H, dt, H, 0.3) * scale
        # eps is an fp32 argument: 1e-40, a subnormal number there, is 71362 * 2^-149, less by 5e-6 of it
        eps = float(torch.tensor(eps, dtype=F32))
        if H > 1:                                     # of one value there is no spread
            check(eff, x, weights(H, F32, H), None, eps=eps)
    if H > 1:                                         # subnormal numbers, whose rstd fp32 does not hold
        x = (rows(5, H, F32, H, 0.3) * 2.0 ** -130).to(dt)
        y, rstd = torch.empty_like(x).cuda(), torch.empty(5, device="cuda")
        eff.layer_norm(x.cuda(), y, eps=0.0, rstd=rstd)
        want, err = B.norm64(x, None, None, 0.0)[:2]
        flat = (x == x[:, :1]).all(1)                 # so few digits are left that two values may be equal: 0 / 0
        assert torch.isnan(y.cpu()[flat]).all() and not flat.all()
        R.assert_within(y[~flat.cuda()], want[~flat], err[~flat], "y")


@pytest.mark.parametrize("H", [512, 8192, 1 << 15])
def test_no_spread(eff, H):
    """Equal values of any size: eps alone is the variance, or the row is 0 / 0."""
    for v in (1.0, 2.0 ** 70, 3.0 * 2.0 ** 125, -2.0 ** 127):
        for eps in (1e-5, 1e-37):
            x = torch.full((3, H), v, dtype=BF, device="cuda")
            y, mean, rstd = torch.full_like(x, 5.0), torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
            eff.layer_norm(x, y, eps=eps, mean=mean, rstd=rstd)
            want = torch.full((3,), eps, device="cuda").double() ** -0.5
            assert not y.any() and (mean == v).all()
            R.assert_within(rstd, want, 4 * B.U * want, "rstd")
        eff.layer_norm(x, y, eps=0.0)
        assert torch.isnan(y).all()


@pytest.mark.parametrize("H", [40, 700, 2048, 8200, 16400])
def test_beside_ordinary_rows(eff, H):
    """Such rows change nothing for the others, in the same workgroup or not; NaN and infinities stay in theirs."""
    x = rows(9, H, F32, H)
    mixed = x.clone()
    mixed[1] *= 1e30
    mixed[3, 5], mixed[4, 0], mixed[7] = float("nan"), float("-inf"), 3e38
    y, y2, mean, rstd = [torch.empty_like(x).cuda() for _ in range(2)] + [torch.empty(9, device="cuda") for _ in range(2)]
    eff.layer_norm(x.cuda(), y)
    eff.layer_norm(mixed.cuda(), y2, mean=mean, rstd=rstd)
    same = [0, 2, 5, 6, 8]
    assert torch.equal(y[same], y2[same])
    assert torch.isnan(y2[3:5]).all() and torch.isnan(mean[3:5]).all() and torch.isnan(rstd[3:5]).all()
    ry, ye, rm, me, rr, re = B.norm64(mixed[1:2], None, None, 1e-5)
    R.assert_within(y2[1:2], ry, ye, "y")
    R.assert_within(mean[1:2], rm[:, 0], me[:, 0], "mean")
    R.assert_within(rstd[1:2], rr[:, 0], re[:, 0], "rstd")
    assert torch.isfinite(y2[7]).all() and torch.isfinite(rstd[7])
    # an eps beyond the scaled squares, too
    x = rows(3, H, F32, H) * 2.0 ** 64
    check(eff, x, None, None, eps=2.0 ** 127)
    check(eff, x, None, None, eps=2.0 ** 100)
