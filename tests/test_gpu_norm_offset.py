"""Layer norm's gradients of rows whose offset is far above their spread, against the definition's own: the statistics that the
forward pass saves are rounded to fp32, and that is all that is lost."""
import pytest
import torch

from tests import block_ref as B
from tests import ops_ref as R

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    return e


def saved(dy, x, w, eps):
    """(dx, bound, dw, bound) of the definition, the bounds with what the saved statistics' own errors add to norm_grad64's.

    A mean off by m and an rstd off by a share q move xh by s = m rstd + q |xh| (1 + q).  dw moves by sum |dy| s; mean(g xh) by
    mean |g| s =: v; dx = rstd (g - mean g - xh mean(g xh)) by q of its terms' magnitudes and (1 + q) rstd (s (a2 + v) + |xh| v)."""
    _, _, mean, me, rstd, re = B.norm64(x, None, None, eps)
    dx, ex, dw, ew, _, _ = B.norm_grad64(dy, x, w, mean[:, 0], rstd[:, 0], None)
    dy, x = dy.double(), x.double()
    xh, g = (x - mean) * rstd, dy * w.double()
    m, q = me, re / rstd                              # their bounds hold the rounding of what is saved
    s = m * rstd + q * xh.abs() * (1 + q)
    v, a1, a2 = (g.abs() * s).mean(1, keepdim=True), g.abs().mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
    ex = ex * (1 + 1e-3) + q * rstd * (g.abs() + a1 + xh.abs() * a2) + (1 + q) * rstd * (s * (a2 + v) + xh.abs() * v)
    return dx, ex, dw, ew * (1 + 1e-3) + (dy.abs() * s).sum(0)


@pytest.mark.parametrize("H", [40, 256, 1000, 4096, 8192, 20000])
@pytest.mark.parametrize("offset,spread", [(1000.0, 1e-2), (-3e4, 1.0), (0.5, 1.0)])
def test_gradients(eff, H, offset, spread):
    T = 6
    g = torch.Generator().manual_seed(H)
    x = (offset + spread * torch.randn(T, H, generator=g, dtype=torch.float64)).to(F32)
    dy, w = torch.randn(T, H, generator=g), 1 + 0.3 * torch.randn(H, generator=g)
    mean, rstd, y = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty(T, H, device="cuda")
    eff.layer_norm(x.cuda(), y, weight=w.cuda(), eps=1e-9, mean=mean, rstd=rstd)
    ry, ye = B.norm64(x, w, None, 1e-9)[:2]
    R.assert_within(y, ry, ye, "y")
    dx, dw = torch.empty(T, H, device="cuda"), torch.empty(H, device="cuda")
    eff.layer_norm_backward(dy.cuda(), x.cuda(), mean, rstd, dx=dx, dw=dw, weight=w.cuda())
    rx, xe, rw, we = saved(dy, x, w, 1e-9)
    R.assert_within(dx, rx, xe, "dx")
    R.assert_within(dw, rw, we, "dw")
    # what the documentation says of the shift: half a step of the mean, 2^-24 of it at most, next to the sums' own error (norm64)
    m64 = B.norm64(x, None, None, 1e-9)[2]
    D, ax = B.depth(H), x.double().abs().mean(1, keepdim=True)
    sums = (D + 6) * B.U * ((x.double() - m64).abs().mean(1, keepdim=True) + (D + 4) * B.U * ax)
    assert ((mean.cpu().double()[:, None] - m64).abs() <= B.U * (m64.abs() + sums) + sums).all()
