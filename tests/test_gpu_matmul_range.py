"""Gradients in fp16 whose dz = dy * act'(z) does not fit fp16, although the gradients do: fp32 or large dy, and small dy
that only the sum brings back.  Against 64 bits.

Bounds.  dz enters the products as fp16 after a power of two that brings the largest of its row (dx) or of its column in a
group (dw) into [2^14, 2^15): an element is off by half a step of its own, 2^-12 of it, and where that is subnormal by
2^-25 / 2^14 = 2^-39 of the largest.  The fp32 sums, functions and the last rounding as in ops_ref."""
import pytest
import torch

from tests import ops_ref as R

pytestmark = pytest.mark.gpu
HF, F32 = torch.float16, torch.float32


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    return e


def powers(g, count, lo, hi):
    return 2.0 ** torch.randint(lo, hi + 1, (count,), generator=g).double()


def dz_of(dy, pre, act):
    dy = dy.double()
    return (dy, dy.abs()) if act == R.NONE else R.dz64(dy, pre.double(), act)


def inputs(m, n, k, act, lo, hi, wscale, counts=None, dy_type=F32, seed=0):
    g = torch.Generator().manual_seed(seed * 31 + m + n + k + act)
    nw = 2 * n if act == R.SWIGLU else n
    lead = (len(counts),) if counts else ()
    x = (torch.randn(m, k, generator=g) * wscale).to(HF)
    w = (torch.randn(*lead, nw, k, generator=g) * wscale).to(HF)
    pre = torch.randn(m, nw, generator=g).to(HF) if act else None
    dy = (torch.randn(m, n, generator=g).double() * powers(g, m, lo, hi)[:, None] * powers(g, n, 0, 3)).to(dy_type)
    off = torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32) if counts else None
    return x, w, pre, dy, off


def run(eff, x, w, pre, dy, off, act):
    dx, dw = torch.full_like(x, 7.0, device="cuda"), torch.full_like(w, 7.0, device="cuda")
    args = dict(dx=dx, dw=dw, act=act, pre=None if pre is None else pre.cuda())
    if off is None:
        eff.matmul_backward(dy.cuda(), x.cuda(), w.cuda(), **args)
    else:
        eff.grouped_matmul_backward(dy.cuda(), x.cuda(), w.cuda(), off.cuda(), **args)
    return dx, dw


def check(x, w, pre, dy, off, act, dx, dw, rows_of_dx=slice(None)):
    m, nw = x.shape[0], w.shape[-2]
    dz, mag = dz_of(dy, pre, act)
    func = R.FUNC * mag if act else torch.zeros_like(mag)
    own = R.half_ulp(HF) * (dz.abs() + func) + func
    xd, wd = x.double(), w.double()
    for e, rows in R.groups_of(off, m):
        we, z, ze, xr = (wd if e is None else wd[e]), dz[rows], own[rows], xd[rows]
        if not len(z):
            assert not dw[e].any()
            continue
        top = (z.abs() + ze)
        zx, zw = ze + 2.0 ** -39 * top.amax(1, keepdim=True), ze + 2.0 ** -39 * top.amax(0, keepdim=True)
        ref = z @ we
        assert float(ref.abs().max()) < 65504
        R.assert_within(dx[rows], ref, zx @ we.abs() + (nw + 8) * R.STEP * ((z.abs() + zx) @ we.abs()), "dx")
        ref = z.t() @ xr
        assert float(ref.abs().max()) < 65504
        R.assert_within(dw if e is None else dw[e], ref, zw.t() @ xr.abs() + (len(z) + 8) * R.STEP * ((z.abs() + zw).t() @ xr.abs()), "dw")


SHAPES = [(1, 8, 16), (3, 5, 7), (40, 24, 32), (70, 136, 72), (300, 264, 136), (1030, 520, 264)]


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("shape", SHAPES)
def test_large_dz(eff, shape, act):
    """Rows of dy of 2^14 to 2^22, in fp32; x and w small."""
    case = inputs(*shape, act, 14, 22, 2.0 ** -17)
    check(*case, act, *run(eff, *case, act))


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("shape", SHAPES)
def test_small_dz(eff, shape, act):
    """Rows of dy of 2^-36 to 2^-24; x and w large, so that the sums are back in range."""
    case = inputs(*shape, act, -36, -24, 2.0 ** 12)
    check(*case, act, *run(eff, *case, act))


def test_fp16_dy_and_a_large_up(eff):
    """dy and the saved sums fit fp16, their product does not."""
    x, w, pre, dy, off = inputs(70, 72, 40, R.SWIGLU, 6, 8, 2.0 ** -12, dy_type=HF)
    pre[:, 72:] *= 1000
    assert float(dz_of(dy, pre, R.SWIGLU)[0].abs().max()) > 65504
    check(x, w, pre, dy, off, R.SWIGLU, *run(eff, x, w, pre, dy, off, R.SWIGLU))


@pytest.mark.parametrize("lo,hi,scale", [(14, 22, 2.0 ** -17), (-36, -24, 2.0 ** 12)])
@pytest.mark.parametrize("counts", [[5], [1, 0, 3, 0, 0, 2], [130, 0, 7], [33] * 40, [300, 1, 257]], ids=str)
@pytest.mark.parametrize("act", [R.NONE, R.SWIGLU])
def test_groups(eff, counts, act, lo, hi, scale):
    for n, k in ((72, 136), (33, 50)):
        case = inputs(sum(counts), n, k, act, lo, hi, scale, counts=counts)
        check(*case, act, *run(eff, *case, act))


def test_one_gradient_only(eff):
    x, w, pre, dy, off = inputs(70, 40, 64, R.GELU, 14, 22, 2.0 ** -17)
    dx, dw = run(eff, x, w, pre, dy, off, R.GELU)
    for want in (("dx",), ("dw",), ("dx", "dbias"), ("dbias",)):
        out = {"dx": torch.full_like(dx, 7.0), "dw": torch.full_like(dw, 7.0), "dbias": torch.full((40,), 7.0, dtype=HF, device="cuda")}
        eff.matmul_backward(dy.cuda(), x.cuda(), w.cuda(), act=R.GELU, pre=pre.cuda(), **{o: out[o] for o in want})
        assert torch.equal(out["dx"], dx if "dx" in want else torch.full_like(dx, 7.0))
        assert torch.equal(out["dw"], dw if "dw" in want else torch.full_like(dw, 7.0))


def test_values_that_are_not_finite(eff):
    """An infinity and a NaN in dy reach their own row of dx and their own columns of dw; the others are as without."""
    x, w, pre, dy, off = inputs(40, 24, 32, R.SILU, 14, 22, 2.0 ** -17)
    clean = run(eff, x, w, pre, dy, off, R.SILU)
    dy = dy.clone()
    dy[3, 5], dy[8, 6] = float("inf"), float("nan")
    dx, dw = run(eff, x, w, pre, dy, off, R.SILU)
    assert not torch.isfinite(dx[3]).any() and torch.isnan(dx[8]).all()
    assert not torch.isfinite(dw[5]).any() and torch.isnan(dw[6]).all()
    keep = [i for i in range(40) if i not in (3, 8)]
    assert torch.equal(dx[keep], clean[0][keep])
    keep = [i for i in range(24) if i not in (5, 6)]
    assert torch.equal(dw[keep], clean[1][keep])


def test_no_rows_and_no_gradient(eff):
    dw = torch.full((16, 32), 3.0, dtype=HF, device="cuda")
    x = torch.empty(0, 32, dtype=HF, device="cuda")
    eff.matmul_backward(torch.empty(0, 16, dtype=F32, device="cuda"), x, torch.ones_like(dw), dx=torch.empty_like(x), dw=dw)
    assert not dw.any()
    x, w, pre, dy, off = inputs(40, 24, 32, R.NONE, 0, 0, 1.0)
    dx, dw = run(eff, x, w, pre, torch.zeros_like(dy), off, R.NONE)
    assert not dx.any() and not dw.any()


def test_replayed_with_other_magnitudes(eff):
    """A captured backward pass, replayed on dy of other sizes: nothing of an earlier replay's scales is left."""
    counts = [20, 0, 47]
    x, w, pre, dy, off = inputs(67, 40, 72, R.SWIGLU, 0, 0, 2.0 ** -10, counts=counts)
    d = [t.cuda() for t in (dy, x, w, off, pre)]
    dx, dw = torch.zeros_like(d[1]), torch.zeros_like(d[2])

    def once():
        eff.grouped_matmul_backward(*d[:4], dx=dx, dw=dw, act=R.SWIGLU, pre=d[4])

    once()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once()
    for shift in (16, -16, 0, 8):
        d[0].copy_((dy * 2.0 ** shift).cuda())
        dx.fill_(7.0)
        dw.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = dx.clone(), dw.clone()
        check(x, w, pre, dy * 2.0 ** shift, off, R.SWIGLU, *got)
        once()
        torch.cuda.synchronize()
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
