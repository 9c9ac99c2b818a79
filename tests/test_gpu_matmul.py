"""Products with bias, activation and residual, dense and grouped, and their gradients, against 64 bits."""
import pytest
import torch

from tests import ops_ref as R

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    return e


def rnd(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def strided(t, pad):
    """The same values on the GPU with `pad` elements (holding NaN) between rows."""
    if not pad:
        return t.cuda()
    big = torch.full(t.shape[:-1] + (t.shape[-1] + pad,), float("nan"), dtype=t.dtype, device="cuda")
    big[..., :t.shape[-1]] = t.cuda()
    return big[..., :t.shape[-1]]


def offsets_of(counts, before=0):
    return torch.tensor([before] + [before + sum(counts[:i + 1]) for i in range(len(counts))], dtype=torch.int32)


def to(t, work):
    """Large references are computed on the GPU, in 64 bits all the same."""
    return t if t is None or work < 10 ** 8 else t.cuda()


def run_forward(eff, m, n, k, dtype=BF, out=None, act=R.NONE, bias=False, residual=False, pre=False, counts=None, pad=0, seed=0,
                before=0):
    g = torch.Generator().manual_seed(seed * 1000003 + m * 7919 + n * 31 + k)
    nw = 2 * n if act == R.SWIGLU else n
    lead = (len(counts),) if counts else ()
    x, w = rnd(g, m, k, dtype=dtype), rnd(g, *lead, nw, k, dtype=dtype, scale=k ** -0.5)
    b = rnd(g, *lead, nw, dtype=dtype) if bias else None
    r = rnd(g, m, n, dtype=dtype) if residual else None
    off = offsets_of(counts, before) if counts else None
    inside = torch.ones(m, dtype=torch.bool) if off is None else (torch.arange(m) >= off[0]) & (torch.arange(m) < off[-1])
    x[~inside] = float("nan")              # rows in no group are not read
    y = strided(torch.full((m, n), 7.0, dtype=out or dtype), pad)
    p = strided(torch.full((m, nw), 7.0, dtype=dtype), pad) if pre else None
    args = dict(bias=None if b is None else b.cuda(), act=act, residual=None if r is None else strided(r, pad), pre=p)
    if off is None:
        eff.matmul(strided(x, pad), strided(w, pad), y, **args)
    else:
        eff.grouped_matmul(strided(x, pad), strided(w, pad), off.cuda(), y, **args)
    torch.cuda.synchronize()
    x = torch.where(inside[:, None], x.float(), 0.0).to(dtype)
    ry, ye, rz, ze = (t.cpu() for t in R.matmul64(*(to(t, m * nw * k) for t in (x, w, b)), act, to(r, m * nw * k), off, n))
    what = "m%d n%d k%d %s act%d" % (m, n, k, dtype, act)
    assert (y[~inside.cuda()] == 7).all(), "rows in no group changed"
    R.assert_within(y[inside.cuda()], ry[inside], ye[inside], what + " y")
    if pre:
        assert (p[~inside.cuda()] == 7).all()
        R.assert_within(p[inside.cuda()], rz[inside], ze[inside], what + " pre")
    if pad:
        assert torch.isnan(y.as_strided((m, pad), (y.stride(0), 1), y.storage_offset() + n)).all(), "written between rows"


SHAPES = [(1, 1, 1), (1, 64, 64), (2, 3, 5), (1, 512, 2560), (16, 640, 256), (17, 129, 100), (33, 66, 72), (64, 64, 32),
          (100, 200, 328), (130, 257, 65), (256, 256, 512), (300, 520, 1032), (513, 384, 192)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("shape", SHAPES)
def test_plain_product(eff, shape, dtype):
    run_forward(eff, *shape, dtype=dtype)


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("shape", [(1, 512, 640), (5, 35, 24), (16, 128, 256), (19, 40, 33), (70, 136, 264), (260, 300, 520)])
def test_epilogues(eff, shape, act):
    run_forward(eff, *shape, act=act, bias=True, residual=True, pre=True)
    run_forward(eff, *shape, dtype=HF, act=act, bias=False, residual=True, pre=False, seed=1)


@pytest.mark.parametrize("shape", [(1, 256, 2048), (7, 8, 8), (40, 256, 512), (200, 96, 136)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_fp32_output(eff, shape, dtype):
    run_forward(eff, *shape, dtype=dtype, out=F32, bias=True)
    run_forward(eff, *shape, dtype=dtype, out=F32, act=R.SWIGLU, residual=True, seed=2)


@pytest.mark.parametrize("pad", [1, 2, 4, 8, 24])
@pytest.mark.parametrize("shape", [(1, 64, 128), (16, 96, 64), (65, 130, 72), (129, 256, 320), (300, 264, 584)])
def test_strides_between_rows(eff, shape, pad):
    run_forward(eff, *shape, act=R.SWIGLU, residual=True, pre=True, pad=pad)
    run_forward(eff, *shape, act=R.GELU, bias=True, pad=pad, dtype=HF)


@pytest.mark.parametrize("shift", [1, 2, 4, 8])
@pytest.mark.parametrize("m", [1, 9, 140])
def test_unaligned_pointers(eff, m, shift):
    n, k = 96, 128
    g = torch.Generator().manual_seed(shift)
    bufs = [torch.zeros(s + 16, dtype=BF, device="cuda") for s in (m * k, n * k, n, m * n, m * n)]
    x, w, b, r = rnd(g, m, k), rnd(g, n, k, scale=0.1), rnd(g, n), rnd(g, m, n)
    views = [buf[shift:shift + t.numel()].view(t.shape) for buf, t in zip(bufs, (x, w, b, r, r))]
    for v, t in zip(views, (x, w, b, r)):
        v.copy_(t)
    eff.matmul(views[0], views[1], views[4], bias=views[2], act=R.SILU, residual=views[3])
    ry, ye, _, _ = R.matmul64(x, w, b, R.SILU, r, None, n)
    R.assert_within(views[4], ry, ye, "unaligned")
    assert (bufs[4][:shift] == 0).all() and (bufs[4][shift + m * n:] == 0).all()


COUNTS = [[0, 0, 0], [5], [1, 0, 3, 0, 0, 2], [0, 64, 1, 63, 65, 0], [130, 0, 7], [3] * 40, [0] * 100 + [9] + [0] * 50, [300, 1, 257]]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "g%d_%d" % (len(c), sum(c)))
@pytest.mark.parametrize("act", [R.NONE, R.SWIGLU])
def test_grouped(eff, counts, act):
    m = sum(counts) + 3       # rows behind the last group
    run_forward(eff, m, 72, 136, act=act, bias=True, residual=True, pre=True, counts=counts)
    run_forward(eff, m, 33, 50, act=act, dtype=HF, counts=counts, pad=1)


@pytest.mark.parametrize("counts", [[4, 0, 9], [70, 200, 3]])
def test_groups_that_begin_late(eff, counts):
    run_forward(eff, sum(counts) + 10, 64, 64, act=R.GELU_TANH, bias=True, counts=counts, before=5)


def test_wide_groups(eff):
    """4096 groups, and offsets that are not sound stay inside the buffers."""
    counts = [i % 3 for i in range(4096)]
    run_forward(eff, sum(counts), 16, 32, counts=counts)
    x, w = torch.ones(8, 16, dtype=BF, device="cuda"), torch.ones(2, 8, 16, dtype=BF, device="cuda")
    for off in ([0, -5, 3], [-7, 100, 2], [2147483647, 0, 8], [0, 8, 2147483647], [8, 4, 0]):
        buf = torch.full((24, 8), 7.0, dtype=BF, device="cuda")
        eff.grouped_matmul(x, w, torch.tensor(off, dtype=torch.int32, device="cuda"), buf[8:16])
        torch.cuda.synchronize()
        assert (buf[:8] == 7).all() and (buf[16:] == 7).all()
        assert ((buf[8:16] == 7) | (buf[8:16] == 16)).all()


def test_residual_in_place_and_broadcast(eff):
    g = torch.Generator().manual_seed(3)
    for m, n, k in ((5, 24, 40), (200, 136, 264)):
        x, w, r = rnd(g, m, k), rnd(g, n, k, scale=0.2), rnd(g, m, n)
        y = r.cuda()
        eff.matmul(x.cuda(), w.cuda(), y, act=R.SILU, residual=y)
        ry, ye, _, _ = R.matmul64(x, w, None, R.SILU, r, None, n)
        R.assert_within(y, ry, ye, "in place")
        row = rnd(g, 1, n)
        eff.matmul(x.cuda(), w.cuda(), y, residual=row.cuda().expand(m, n))
        ry, ye, _, _ = R.matmul64(x, w, None, R.NONE, row.expand(m, n), None, n)
        R.assert_within(y, ry, ye, "broadcast residual")
        xr = rnd(g, 1, k)
        eff.matmul(xr.cuda().expand(m, k), w.cuda(), y)
        ry, ye, _, _ = R.matmul64(xr.expand(m, k), w, None, R.NONE, None, None, n)
        R.assert_within(y, ry, ye, "broadcast x")


def test_no_rows(eff):
    x, w = torch.empty(0, 32, dtype=BF, device="cuda"), torch.ones(16, 32, dtype=BF, device="cuda")
    eff.matmul(x, w, torch.empty(0, 16, dtype=BF, device="cuda"))
    dw, db = torch.full((16, 32), 3.0, dtype=BF, device="cuda"), torch.full((16,), 3.0, dtype=BF, device="cuda")
    eff.matmul_backward(torch.empty(0, 16, dtype=BF, device="cuda"), x, w, dx=torch.empty_like(x), dw=dw, dbias=db)
    assert (dw == 0).all() and (db == 0).all()


def test_values_that_are_not_finite_stay_in_their_row(eff):
    g = torch.Generator().manual_seed(4)
    for m, n, k in ((3, 64, 64), (150, 128, 96)):
        x, w = rnd(g, m, k), rnd(g, n, k)
        x[1, 5], x[2, 6] = float("nan"), float("inf")
        y = torch.empty(m, n, dtype=BF, device="cuda")
        eff.matmul(x.cuda(), w.cuda(), y)
        ref = (x.double() @ w.double().t())
        assert torch.isnan(y[1]).all() and (torch.isinf(y[2].cpu()) == torch.isinf(ref[2])).all()
        keep = [i for i in range(m) if i not in (1, 2)]
        assert torch.isfinite(y[keep]).all()


def test_saturated_activations(eff):
    """Sums far out on both sides: the activations reach 0 and the identity, their gradients 0 and 1, with no NaN."""
    z = torch.tensor([-1e30, -3e4, -100.0, -20.0, 0.0, 20.0, 100.0, 3e4, 1e30], dtype=torch.float32).to(BF)
    x, w = torch.zeros(len(z), 8, dtype=BF), torch.zeros(16, 8, dtype=BF)
    x[:, 0], w[:, 0] = z, 1.0
    for act in range(5):
        n = 8 if act == R.SWIGLU else 16
        if act == R.SWIGLU:
            w[8:] = 0.0
            w[8:, 1], x[:, 1] = 1.0, 1.0     # up = 1
        y, pre = torch.empty(len(z), n, dtype=BF, device="cuda"), torch.empty(len(z), 16, dtype=BF, device="cuda")
        eff.matmul(x.cuda(), w.cuda(), y, act=act, pre=pre)
        dx = torch.empty_like(x, device="cuda")
        dy = torch.ones_like(y)
        eff.matmul_backward(dy, x.cuda(), w.cuda(), dx=dx, act=act, pre=pre)
        assert torch.isfinite(y).all() and torch.isfinite(dx).all(), act
        if act:
            assert (y[:3].abs() < 1e-30).all(), act
        assert (y[6:, 0].cpu() == z[6:]).all(), act
        lo, hi = dx[0, 0].item(), dx[-1, 0].item()
        assert hi == n and (act == 0 or lo == 0), (act, lo, hi)


# ---- gradients

def run_backward(eff, m, n, k, dtype=BF, act=R.NONE, counts=None, pad=0, dy32=False, want=("dx", "dw", "dbias"), before=0):
    g = torch.Generator().manual_seed(m * 7919 + n * 31 + k + act)
    nw = 2 * n if act == R.SWIGLU else n
    lead = (len(counts),) if counts else ()
    x, w = rnd(g, m, k, dtype=dtype), rnd(g, *lead, nw, k, dtype=dtype, scale=k ** -0.5)
    dy = rnd(g, m, n, dtype=F32 if dy32 else dtype)
    pre = rnd(g, m, nw, dtype=dtype) if act else None
    off = offsets_of(counts, before) if counts else None
    inside = torch.ones(m, dtype=torch.bool) if off is None else (torch.arange(m) >= off[0]) & (torch.arange(m) < off[-1])
    x[~inside] = float("nan")
    dy[~inside] = float("nan")
    out = {"dx": strided(torch.full((m, k), 7.0, dtype=dtype), pad), "dw": strided(torch.full(lead + (nw, k), 7.0, dtype=dtype), pad),
           "dbias": torch.full(lead + (nw,), 7.0, dtype=dtype, device="cuda")}
    args = dict(act=act, pre=None if pre is None else strided(pre, pad), **{o: out[o] for o in want})
    if off is None:
        eff.matmul_backward(strided(dy, pad), strided(x, pad), strided(w, pad), **args)
    else:
        eff.grouped_matmul_backward(strided(dy, pad), strided(x, pad), strided(w, pad), off.cuda(), **args)
    torch.cuda.synchronize()
    xd, wd, dyd = torch.where(inside[:, None], x.double(), 0.0), w.double(), torch.where(inside[:, None], dy.double(), 0.0)
    dz, mag = dz64(dyd, pre, act)
    step = R.half_ulp(dtype) if act or dy32 else 0.0
    # what dz may be off by where it enters the products (its rounding, the functions), and before it
    func = R.FUNC * mag if act else torch.zeros_like(mag)
    dze = func + step * (dz.abs() + func) + (R.tiny(dtype) if step else 0.0)
    what = "m%d n%d k%d act%d %s" % (m, n, k, act, dtype)
    ref = {"dx": torch.zeros(m, k, dtype=torch.float64), "dw": torch.zeros(lead + (nw, k), dtype=torch.float64),
           "dbias": torch.zeros(lead + (nw,), dtype=torch.float64)}
    err = {o: torch.zeros_like(v) for o, v in ref.items()}
    xd, wd, dz, dze, func = (to(t, m * nw * k) for t in (xd, wd, dz, dze, func))
    for e, rows in R.groups_of(off, m):
        z, ze, xr = dz[rows], dze[rows], xd[rows]
        we = wd if e is None else wd[e]
        at = slice(None) if e is None else e
        cnt = z.shape[0]
        ref["dx"][rows] = z @ we
        err["dx"][rows] = ze @ we.abs() + (nw + 8) * R.STEP * ((z.abs() + ze) @ we.abs())
        ref["dw"][at] = z.t() @ xr
        err["dw"][at] = ze.t() @ xr.abs() + (cnt + 8) * R.STEP * ((z.abs() + ze).t() @ xr.abs())
        ref["dbias"][at] = z.sum(0)
        err["dbias"][at] = func[rows].sum(0) + (cnt + 8) * R.STEP * (z.abs() + func[rows]).sum(0)
    for o in want:
        got = out[o]
        if o == "dx":
            assert (got[~inside.cuda()] == 7).all()
            R.assert_within(got[inside.cuda()], ref[o][inside], err[o][inside], what + " dx")
        else:
            R.assert_within(got, ref[o], err[o], what + " " + o)
    for o in set(out) - set(want):
        assert (out[o] == 7).all()


def dz64(dy, pre, act):
    if act == R.NONE:
        return dy, dy.abs()
    return R.dz64(dy, pre.double(), act)


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("shape", [(1, 8, 16), (3, 5, 7), (16, 64, 128), (65, 66, 72), (130, 128, 256), (257, 96, 520)])
def test_gradients(eff, shape, act):
    run_backward(eff, *shape, act=act)
    run_backward(eff, *shape, act=act, dtype=HF, pad=8)


@pytest.mark.parametrize("shape", [(1, 256, 64), (40, 24, 48), (300, 256, 136)])
def test_gradients_of_fp32_outputs(eff, shape):
    run_backward(eff, *shape, dy32=True)
    run_backward(eff, *shape, act=R.SWIGLU, dy32=True, dtype=HF)


@pytest.mark.parametrize("want", [("dx",), ("dw",), ("dbias",), ("dx", "dbias")])
@pytest.mark.parametrize("act", [R.NONE, R.GELU])
def test_some_gradients_only(eff, want, act):
    run_backward(eff, 70, 40, 64, act=act, want=want)


@pytest.mark.parametrize("pad", [1, 3, 8])
def test_gradients_of_strided_matrices(eff, pad):
    run_backward(eff, 70, 40, 72, act=R.SWIGLU, pad=pad)
    run_backward(eff, 70, 40, 72, pad=pad)


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "g%d_%d" % (len(c), sum(c)))
@pytest.mark.parametrize("act", [R.NONE, R.SWIGLU])
def test_grouped_gradients(eff, counts, act):
    m = sum(counts) + 2
    run_backward(eff, m, 40, 72, act=act, counts=counts)
    run_backward(eff, m, 35, 50, act=act, counts=counts, dtype=HF, before=2)


@pytest.mark.parametrize("act", range(5))
def test_gradients_against_differences(eff, act):
    """dx, dw and dbias against central differences of the 64-bit forward (h = 2^-12: the third derivative's term is
    below h^2 times the sums of magnitudes, 6e-8, under the 16-bit roundings that the bound counts)."""
    m, n, k, h = 4, 6, 8, 2.0 ** -12
    g = torch.Generator().manual_seed(act)
    nw = 12 if act == R.SWIGLU else 6
    x, w, b = (torch.randint(-8, 9, s, generator=g).double() / 8 for s in ((m, k), (nw, k), (nw,)))
    c = torch.randint(-4, 5, (m, n), generator=g).double() / 4

    def loss(x, w, b):
        return float((R.act64(x @ w.t() + b, act) * c).sum())

    pre = (x @ w.t() + b)
    pre16 = pre.to(HF)
    assert (pre16.double() == pre).all()      # small grid: exact in fp16
    dx, dw, db = (torch.empty(s, dtype=HF, device="cuda") for s in ((m, k), (nw, k), (nw,)))
    eff.matmul_backward(c.to(HF).cuda(), x.to(HF).cuda(), w.to(HF).cuda(), dx=dx, dw=dw, dbias=db, act=act, pre=pre16.cuda())
    dz, _ = R.dz64(c, pre, act) if act else (c, None)
    mags = {0: dz.abs() @ w.abs(), 1: dz.abs().t() @ x.abs(), 2: dz.abs().sum(0)}
    for i, (v, got) in enumerate(zip((x, w, b), (dx, dw, db))):
        num = torch.zeros_like(v)
        for j in range(v.numel()):
            args = [x, w, b]
            up, dn = v.clone(), v.clone()
            up.view(-1)[j] += h
            dn.view(-1)[j] -= h
            num.view(-1)[j] = (loss(*[up if a is v else a for a in args]) - loss(*[dn if a is v else a for a in args])) / (2 * h)
        lim = (R.half_ulp(HF) + 2e-6) * (mags[i] + num.abs()) + 64 * h * h + R.tiny(HF)
        assert ((got.cpu().double() - num).abs() <= lim).all(), i


# Sizes at which each tile (256 x 256, 128 x 256, 128 x 128, 64 x 128) is taken, some with k split; none is a multiple of its
# tile.  Every tile in every layout, whole and split: matmul_paths.
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("shape", [(2051, 4104, 1032), (2051, 2056, 4104), (2051, 1032, 4104), (1030, 1032, 4104), (2051, 2056, 136),
                                   (2051, 4104, 136)])
def test_every_tile(eff, shape, dtype):
    m, n, k = shape
    run_forward(eff, m, n, k, dtype=dtype, residual=True)
    run_forward(eff, m, n // 2, k, dtype=dtype, act=R.SWIGLU, bias=True, pre=True)


@pytest.mark.parametrize("act", [R.NONE, R.SWIGLU])
@pytest.mark.parametrize("shape", [(1030, 2056, 4104), (4101, 2056, 2056), (3077, 4104, 136), (1030, 4872, 4104), (2051, 1032, 4104),
                                   (4900, 1032, 4104), (4101, 3080, 136)])
def test_every_tile_of_the_gradients(eff, shape, act):
    m, n, k = shape
    run_backward(eff, m, n if act == R.NONE else n // 2, k, act=act)


@pytest.mark.parametrize("m,n,k,groups", [(4101, 2056, 1032, 2), (500, 2056, 136, 40), (2051, 2056, 136, 2), (4101, 1032, 2056, 2),
                                          (20000, 520, 136, 2), (4101, 520, 2056, 2)])
def test_every_tile_of_the_groups(eff, m, n, k, groups):
    g = torch.Generator().manual_seed(m)
    cut = sorted(torch.randint(0, m - 4, (groups - 1,), generator=g).tolist())
    counts = [b - a for a, b in zip([0] + cut, cut + [m - 5])]
    run_forward(eff, m, n, k, counts=counts, bias=True)
    run_forward(eff, m, n // 2, k, counts=counts, act=R.SWIGLU, dtype=HF)
    run_backward(eff, m, n, k, counts=counts)
    run_backward(eff, m, n // 2, k, counts=counts, act=R.SWIGLU, want=("dx", "dw"))


@pytest.mark.parametrize("shape", [(2050, 2051, 133), (40, 515, 2563), (1, 512, 2561), (20, 33, 1001)])
def test_odd_sizes(eff, shape):
    """Rows that are no whole vectors: the operands are packed first."""
    run_forward(eff, *shape, act=R.SILU, bias=True, residual=True, pre=True)
    run_backward(eff, *shape, act=R.GELU)
    run_backward(eff, *shape)
    m, n, k = shape
    run_forward(eff, m * 3, n, k, counts=[m, 2 * m], act=R.SWIGLU)


def test_outputs_larger_than_the_caches(eff):
    """Stored past them: 256 MiB and more of y and of dw."""
    run_forward(eff, 16400, 8200, 40, residual=True)
    run_backward(eff, 300, 1040, 2072, counts=[30] * 8 + [0] * 60, want=("dw",))


# ---- how it is used

def test_large_offsets(eff):
    """Rows and weights further than 2^31 elements from the first."""
    m, n, k, ld = 40, 24, 64, (1 << 26) + 8
    g = torch.Generator().manual_seed(9)
    x, w = rnd(g, m, k), rnd(g, 2, n, k, scale=0.2)
    buf = torch.empty(m * ld, dtype=BF, device="cuda")
    xv = buf.as_strided((m, k), (ld, 1))
    yv = buf.as_strided((m, n), (ld, 1), 128)
    xv.copy_(x)
    yv.zero_()
    eff.matmul(xv, w[0].cuda(), yv)
    ry, ye, _, _ = R.matmul64(x, w[0], None, 0, None, None, n)
    R.assert_within(yv, ry, ye, "dense, far rows")
    wv = buf.as_strided((2, n, k), (1 << 31, k, 1), 512)
    wv.copy_(w)
    xv.copy_(x)
    off = torch.tensor([0, 5, m], dtype=torch.int32)
    eff.grouped_matmul(xv, wv, off.cuda(), yv)
    ry, ye, _, _ = R.matmul64(x, w, None, 0, None, off, n)
    R.assert_within(yv, ry, ye, "grouped, far weights")
    del xv, yv, wv, buf
    torch.cuda.empty_cache()


def test_streams_and_repeats(eff):
    """Calls on two streams at once and repeated calls give the same bits."""
    g = torch.Generator().manual_seed(5)
    cases = []
    for m, n, k in ((1, 512, 2560), (24, 96, 1024), (300, 264, 520)):
        x, w = rnd(g, m, k).cuda(), rnd(g, 2 * n, k, scale=0.05).cuda()
        cases.append((x, w, torch.empty(m, n, dtype=BF, device="cuda"), torch.empty(m, 2 * n, dtype=BF, device="cuda")))
    for x, w, y, p in cases:
        eff.matmul(x, w, y, act=R.SWIGLU, pre=p)
    torch.cuda.synchronize()
    first = [(y.clone(), p.clone()) for _, _, y, p in cases]
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for i in range(9):
        x, w, y, p = cases[i % 3]
        s = streams[i % 2]
        s.wait_stream(torch.cuda.current_stream())
        y2, p2, dx, dw = torch.empty_like(y), torch.empty_like(p), torch.empty_like(x), torch.empty_like(w)
        eff.matmul(x, w, y2, act=R.SWIGLU, pre=p2, stream=s)
        eff.matmul_backward(y2, x, w, dx=dx, dw=dw, act=R.SWIGLU, pre=p2, stream=s if i % 4 else s.cuda_stream)
        outs.append((i % 3, y2, p2, dx, dw))
    torch.cuda.synchronize()
    grads = {}
    for c, y2, p2, dx, dw in outs:
        assert torch.equal(y2, first[c][0]) and torch.equal(p2, first[c][1])
        if c in grads:
            assert torch.equal(dx, grads[c][0]) and torch.equal(dw, grads[c][1])
        grads[c] = (dx, dw)


def test_captured_and_replayed(eff):
    """Forward and backward in one graph, replayed on new inputs with eager work between, equal the eager calls."""
    g = torch.Generator().manual_seed(6)
    for m, n, k in ((1, 256, 1024), (40, 128, 256), (300, 264, 512)):
        counts = [m // 2, 0, m - m // 2]
        off = offsets_of(counts).cuda()
        w, b = rnd(g, 3, 2 * n, k, scale=0.05).cuda(), rnd(g, 3, 2 * n).cuda()
        x, dy = rnd(g, m, k).cuda(), rnd(g, m, n).cuda()

        def both():
            y, p = torch.zeros(m, n, dtype=BF, device="cuda"), torch.zeros(m, 2 * n, dtype=BF, device="cuda")
            dx, dw, db = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(b)
            eff.grouped_matmul(x, w, off, y, bias=b, act=R.SWIGLU, pre=p)
            eff.grouped_matmul_backward(dy, x, w, off, dx=dx, dw=dw, dbias=db, act=R.SWIGLU, pre=p)
            q = torch.zeros(m, n, dtype=F32, device="cuda")
            eff.matmul(x, w[0, :n], q, act=R.SILU)
            return y, p, dx, dw, db, q

        both()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = both()
        for i in range(4):
            x.copy_(rnd(g, m, k).cuda())
            dy.copy_(rnd(g, m, n).cuda())
            graph.replay()
            torch.cuda.synchronize()
            got = [o.clone() for o in outs]
            want = both()
            torch.cuda.synchronize()
            for a, c in zip(got, want):
                assert torch.equal(a, c), (m, i)


def test_two_threads(eff):
    """Calls from two threads at once, each on a stream of its own, give what one thread gives."""
    import threading
    g = torch.Generator().manual_seed(7)
    x, w = rnd(g, 200, 264).cuda(), rnd(g, 528, 264, scale=0.06).cuda()

    def once(stream):
        y, p = torch.empty(200, 264, dtype=BF, device="cuda"), torch.empty(200, 528, dtype=BF, device="cuda")
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        eff.matmul(x, w, y, act=R.SWIGLU, pre=p, stream=stream)
        eff.matmul_backward(y, x, w, dx=dx, dw=dw, act=R.SWIGLU, pre=p, stream=stream)
        return y, p, dx, dw

    want = once(None)
    torch.cuda.synchronize()
    got, failed = [], []

    def work():
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                outs = [once(None) for _ in range(20)]
            s.synchronize()
            got.extend(outs)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and len(got) == 40
    for outs in got:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
