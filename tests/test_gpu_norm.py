"""Layer norm and its gradients against 64 bits (tests/block_ref.py)."""
import pytest
import torch

from tests import block_ref as B
from tests import ops_ref as R

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    return e


def rows(T, H, dt, seed, offset=0.3, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, H, generator=g) * scale + offset).to(dt)


def weights(H, wt, seed, zero=0.0):
    g = torch.Generator().manual_seed(1000 + seed)
    return (torch.randn(H, generator=g) * 0.3 + 1 - zero).to(wt)


def check(eff, x, w, b, eps=1e-5):
    T, H = x.shape
    y, mean, rstd = torch.full_like(x, NAN).cuda(), torch.full((T,), NAN, device="cuda"), torch.full((T,), NAN, device="cuda")
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    eff.layer_norm(x.cuda(), y, weight=cu(w), bias=cu(b), eps=eps, mean=mean, rstd=rstd)
    ry, ye, rm, me, rr, re = B.norm64(x, w, b, eps)
    R.assert_within(y, ry, ye, "y")
    R.assert_within(mean, rm[:, 0], me[:, 0], "mean")
    R.assert_within(rstd, rr[:, 0], re[:, 0], "rstd")
    return y, mean, rstd


def check_grad(eff, dy, x, w, residual, wt, eps=1e-5):
    T, H = x.shape
    _, _, mean, _, rstd, _ = B.norm64(x, w, None, eps)
    mean, rstd = mean[:, 0].float(), rstd[:, 0].float()
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    dx = torch.full_like(x, NAN).cuda()
    dw, db = torch.full((H,), NAN, dtype=wt, device="cuda"), torch.full((H,), NAN, dtype=wt, device="cuda")
    eff.layer_norm_backward(dy.cuda(), x.cuda(), mean.cuda(), rstd.cuda(), dx=dx, dw=dw, db=db, weight=cu(w), residual=cu(residual))
    rx, xe, rw, we, rb, be = B.norm_grad64(dy, x, w, mean, rstd, residual)
    R.assert_within(dx, rx, xe, "dx")
    R.assert_within(dw, rw, we, "dw")
    R.assert_within(db, rb, be, "db")
    return dx, dw, db


# every shape of the row kernels, whole vectors and not, the last vector and the one past it
LENGTHS = [1, 2, 7, 8, 33, 256, 257, 512, 520, 1000, 1025, 2048, 2056, 2560, 4096, 4097, 4104, 8192, 8200, 16384, 16385, 16392, 40001]


@pytest.mark.parametrize("H", LENGTHS)
@pytest.mark.parametrize("dt,wt", [(BF, BF), (BF, F32), (HF, HF), (HF, F32), (F32, F32)])
def test_rows(eff, H, dt, wt):
    for T in (1, 5):
        check(eff, rows(T, H, dt, H + T), weights(H, wt, H), weights(H, wt, H + 1, 1.0) if T == 5 else None)


@pytest.mark.parametrize("H", LENGTHS)
@pytest.mark.parametrize("dt,wt", [(BF, BF), (BF, F32), (HF, HF), (HF, F32), (F32, F32)])
def test_gradients(eff, H, dt, wt):
    for T in (1, 6):
        dy, x = rows(T, H, dt, H, 0.0), rows(T, H, dt, H + T)
        check_grad(eff, dy, x, weights(H, wt, H), rows(T, H, dt, H + 9) if T == 6 else None, wt)


@pytest.mark.parametrize("T,H", [(513, 520), (1500, 257), (2100, 64), (700, 4096), (70, 16400), (600, 16401)])
def test_gradients_over_many_rows(eff, T, H):
    for dt, wt in ((BF, F32), (F32, F32)):
        check_grad(eff, rows(T, H, dt, T, 0.1), rows(T, H, dt, H), weights(H, wt, H), None, wt)


def test_without_weights(eff):
    for dt in (BF, F32):
        x = rows(9, 320, dt, 1)
        check(eff, x, None, None)
        check(eff, x, None, weights(320, F32, 2))
        check_grad(eff, rows(9, 320, dt, 3), x, None, None, F32)
        check_grad(eff, rows(9, 320, dt, 3), x, None, None, dt)


def test_offset_far_above_the_spread(eff):
    """What the first mean rounds away the deviations put right: the spread of fp32 rows around 1000 keeps its digits."""
    for H in (256, 4096, 40000):
        g = torch.Generator().manual_seed(H)
        x = (1000 + 1e-2 * torch.randn(4, H, generator=g)).float()
        check(eff, x, None, None, eps=1e-12)
    x = torch.full((3, 640), 7.25, dtype=BF)          # no spread at all: eps alone
    y, mean, rstd = check(eff, x, None, None)
    assert (y == 0).all() and (mean == 7.25).all()


def test_strides_and_alignment(eff):
    """Rows apart, broadcast, and beginning at odd places; what lies between output rows stays."""
    big = rows(12, 700, BF, 3).cuda()
    w, b = weights(513, BF, 1), weights(513, BF, 2)
    for off, H in ((0, 512), (1, 512), (3, 513), (8, 504)):
        x = big[::2, off:off + H]
        y = torch.full((6, 640), 5.0, dtype=BF, device="cuda")
        wv = torch.zeros(514, dtype=BF)
        wv[1:1 + H] = w[:H]
        wd = wv.cuda()[1:1 + H]                          # weights at an odd place
        eff.layer_norm(x, y[:, off:off + H], weight=wd, bias=b[:H].cuda())
        ry, ye = B.norm64(x.cpu(), w[:H], b[:H], 1e-5)[:2]
        R.assert_within(y[:, off:off + H], ry, ye, "y")
        assert (y[:, :off] == 5).all() and (y[:, off + H:] == 5).all()
        mean, rstd = [t[:, 0].float().cuda() for t in B.norm64(x.cpu(), None, None, 1e-5)[2::2]]
        dy, res = rows(1, H, BF, 4).cuda().expand(6, H), rows(1, H, BF, 5).cuda().expand(6, H)
        dx, dw, db = torch.full((6, 640), 5.0, dtype=BF, device="cuda"), torch.empty(H, dtype=BF, device="cuda"), torch.empty(H, dtype=BF, device="cuda")
        eff.layer_norm_backward(dy, x, mean, rstd, dx=dx[:, off:off + H], dw=dw, db=db, weight=wd, residual=res)
        rx, xe, rw, we, rb, be = B.norm_grad64(dy.cpu(), x.cpu(), w[:H], mean.cpu(), rstd.cpu(), res.cpu())
        R.assert_within(dx[:, off:off + H], rx, xe, "dx")
        R.assert_within(dw, rw, we, "dw")
        R.assert_within(db, rb, be, "db")
        assert (dx[:, :off] == 5).all() and (dx[:, off + H:] == 5).all()


def test_each_output_alone(eff):
    T, H = 300, 264
    dy, x, w = rows(T, H, BF, 1), rows(T, H, BF, 2), weights(H, BF, 3)
    dx, dw, db = check_grad(eff, dy, x, w, None, BF)
    mean, rstd = [t[:, 0].float().cuda() for t in B.norm64(x, None, None, 1e-5)[2::2]]
    for name, want in (("dx", dx), ("dw", dw), ("db", db)):
        got = torch.full_like(want, NAN)
        eff.layer_norm_backward(dy.cuda(), x.cuda(), mean, rstd, weight=w.cuda(), **{name: got})
        assert torch.equal(got, want), name
    y, y2 = torch.empty_like(x).cuda(), torch.empty_like(x).cuda()
    eff.layer_norm(x.cuda(), y)
    eff.layer_norm(x.cuda(), y2, mean=torch.empty(T, device="cuda"))
    assert torch.equal(y, y2)


def test_no_rows(eff):
    x = torch.empty(0, 96, dtype=BF, device="cuda")
    none = torch.empty(0, device="cuda")
    eff.layer_norm(x, torch.empty_like(x), mean=none, rstd=none.clone())
    dw, db = torch.ones(96, dtype=BF, device="cuda"), torch.ones(96, dtype=BF, device="cuda")
    eff.layer_norm_backward(x, x, none, none, dx=torch.empty_like(x), dw=dw, db=db)
    assert not dw.any() and not db.any()


def test_values_that_are_no_numbers_stay_in_their_row(eff):
    for H in (96, 5000, 20000):
        x = rows(5, H, F32, H)
        x[1, 3], x[3, H - 1] = float("inf"), NAN
        y, mean, rstd = torch.empty_like(x).cuda(), torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
        eff.layer_norm(x.cuda(), y, mean=mean, rstd=rstd)
        ok = [0, 2, 4]
        ry, ye = B.norm64(x[ok], None, None, 1e-5)[:2]
        R.assert_within(y[ok], ry, ye, "y")
        assert torch.isnan(y[[1, 3]]).all() and torch.isnan(rstd[[1, 3]]).all()


def test_the_gradients_are_the_formulas_derivatives():
    """The reference itself: against autograd of the definition, and against differences."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(3, 7, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(7, generator=g, dtype=torch.float64, requires_grad=True)
    b = torch.randn(7, generator=g, dtype=torch.float64, requires_grad=True)
    f = lambda x, w, b: (x - x.mean(1, keepdim=True)) * (((x - x.mean(1, keepdim=True)) ** 2).mean(1, keepdim=True) + 1e-5) ** -0.5 * w + b  # noqa: E731
    assert torch.autograd.gradcheck(f, (x, w, b))
    dy = torch.randn(3, 7, generator=g, dtype=torch.float64)
    want = torch.autograd.grad(f(x, w, b), (x, w, b), dy)
    with torch.no_grad():
        mean = x.mean(1)
        rstd = (x.var(1, unbiased=False) + 1e-5) ** -0.5
        got = B.norm_grad64(dy, x, w, mean, rstd, None)[::2]
    for a, c in zip(got, want):
        torch.testing.assert_close(a, c, rtol=1e-11, atol=1e-11)


def test_large_and_repeated(eff):
    """Past 2^31 elements of x, and the same bits from the same call."""
    T, H = 8192, 4096
    x, dy = torch.randn(T, H, device="cuda", dtype=BF), torch.randn(T, H, device="cuda", dtype=BF)
    mean, rstd, y = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(x)
    eff.layer_norm(x, y, mean=mean, rstd=rstd)
    outs = []
    for _ in range(2):
        dx, dw, db = torch.empty_like(x), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
        eff.layer_norm_backward(dy, x, mean, rstd, dx=dx, dw=dw, db=db)
        outs.append((dx, dw, db))
    assert all(torch.equal(a, c) for a, c in zip(*outs))
    xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    mag = (dy.double() * xh).abs().sum(0)
    R.assert_within(outs[0][1], (dy.double() * xh).sum(0), (T // 256 + 72) * B.U * mag, "dw")
    del xh, mag, outs, dx, dw, db, y
    torch.cuda.empty_cache()
    big = torch.empty((1 << 20) + 3, 2056, dtype=BF, device="cuda")
    for at in range(0, big.shape[0], 1 << 18):
        big[at:at + (1 << 18)].normal_()
    out = torch.empty_like(big)
    eff.layer_norm(big, out)
    for r in (0, 1 << 19, big.shape[0] - 1):
        ry, ye = B.norm64(big[r:r + 1].cpu(), None, None, 1e-5)[:2]
        R.assert_within(out[r:r + 1], ry, ye, "row %d" % r)
    del big, out
    torch.cuda.empty_cache()
