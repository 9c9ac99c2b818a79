"""Microscaled 4-bit rows, bit for bit, and the products of such operands against 64 bits."""
import itertools

import pytest
import torch

from tests import block_ref as B
from tests import ops_ref as R
from tests.matmul_paths import group_sizes
from tests.mx4_paths import ONE_ROW_WIDE, PATHS

pytestmark = pytest.mark.gpu
BF, HF, F32, I32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.uint8
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    return e


def empty_rows(eff, *shape):
    cb, sb = eff.mx4_row_bytes(shape[-1])
    return (torch.full((*shape[:-1], cb), 0xAA, dtype=U8, device="cuda"), torch.full((*shape[:-1], sb), 0xAA, dtype=U8, device="cuda"))


def quantised(eff, x):
    c, s = empty_rows(eff, *x.shape)
    eff.mx4_quantize(x, c, s)
    return c, s


def check_rows(eff, x):
    c, s = quantised(eff, x.cuda())
    rc, rs = B.quantise(x)
    assert torch.equal(s.cpu(), rs), "scales"
    assert torch.equal(c.cpu(), B.pack(rc)), "codes"
    want = B.values(c.cpu(), s.cpu())[:, :x.shape[1]]
    for t in (BF, HF, F32):
        y = torch.full(x.shape, NAN, dtype=t, device="cuda")
        eff.mx4_dequantize(c, s, y)
        w = want.to(t)
        assert torch.equal(torch.isnan(y.cpu()), torch.isnan(w)) and torch.equal(y.cpu().nan_to_num(7.0, INF, -INF), w.nan_to_num(7.0, INF, -INF)), t
    return c, s


@pytest.mark.parametrize("m,k", [(1, 1), (1, 31), (2, 32), (3, 33), (1, 127), (5, 128), (4, 129), (7, 640), (3, 1000), (16, 2560), (9, 2563)])
@pytest.mark.parametrize("dt", [BF, HF, F32])
def test_rows(eff, m, k, dt):
    g = torch.Generator().manual_seed(m * k)
    check_rows(eff, (torch.randn(m, k, generator=g) * torch.exp(3 * torch.randn(m, k, generator=g))).to(dt))


@pytest.mark.parametrize("dt", [BF, HF])
def test_every_16_bit_value(eff, dt):
    """Each of the 65536 values alone in its block (its own scale), and under a larger one (another's scale), zeros, both
    signs, subnormal numbers, infinities and NaN among them."""
    v = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(dt)
    alone = torch.zeros(1 << 16, 32, dtype=dt)
    alone[:, 13] = v
    check_rows(eff, alone.view(-1, 128))
    pair = torch.stack([v, torch.roll(v, 97)], 1)
    both = torch.zeros(1 << 16, 32, dtype=dt)
    both[:, 3:5] = pair
    check_rows(eff, both.view(-1, 128))


def test_every_code_at_every_scale(eff):
    """Exact in bf16 and fp32, rounded once in fp16; scale 255 is NaN whatever the code."""
    c = torch.arange(256, dtype=U8).view(-1, 16).repeat(256, 1)     # 32 values each
    s = torch.arange(256, dtype=U8).repeat_interleave(16)
    codes, scales = c.reshape(-1, 64).cuda(), s.reshape(-1, 4).cuda()
    want = B.values(codes.cpu(), scales.cpu())
    for t in (BF, HF, F32):
        y = torch.empty(codes.shape[0], 128, dtype=t, device="cuda")
        eff.mx4_dequantize(codes, scales, y)
        w = want.to(t)
        assert torch.equal(torch.isnan(y.cpu()), torch.isnan(want)), t
        assert torch.equal(y.cpu().nan_to_num(7.0, INF, -INF), w.nan_to_num(7.0, INF, -INF)), t


def test_rounding_at_the_borders(eff):
    """Midpoints and their neighbours in fp32, under scales from the least to the largest."""
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0])
    near = torch.cat([torch.nextafter(mids, torch.tensor(0.0)), mids, torch.nextafter(mids, torch.tensor(9.0))])
    for e in (-126, -120, -20, 0, 20, 125):
        x = torch.zeros(2, 128)
        x[0, :27], x[1, :27] = near, -near
        x[:, 31] = 4.0                                # keeps the exponent at 0 where 7 and its neighbours are not there
        x[:, 32] = 7.9999995
        check_rows(eff, torch.ldexp(x, torch.tensor(e)))
    tiny = torch.zeros(1, 128)
    tiny[0, :4] = torch.tensor([1e-45, 1e-40, 2.0 ** -128, 2.0 ** -127])
    tiny[0, 32:36] = torch.tensor([1e-45, 3e-45, -1e-45, 0.0])
    check_rows(eff, tiny)


def test_stacks_strides_and_alignment(eff):
    g = torch.Generator().manual_seed(4)
    x3 = torch.randn(3, 5, 200, generator=g).to(BF)
    c3, s3 = quantised(eff, x3.cuda())
    c2, s2 = quantised(eff, x3.view(15, 200).cuda())
    assert torch.equal(c3.view(15, -1), c2) and torch.equal(s3.view(15, -1), s2)
    y3 = torch.empty_like(x3).cuda()
    eff.mx4_dequantize(c3, s3, y3)
    assert torch.equal(y3.view(15, 200).cpu().double(), B.values(c2.cpu(), s2.cpu())[:, :200])
    big = torch.randn(10, 400, generator=g).to(BF).cuda()
    for off, k in ((0, 256), (1, 256), (3, 131), (8, 136)):
        x = big[::2, off:off + k]
        cb, sb = eff.mx4_row_bytes(k)
        c, s = torch.full((5, cb + 16), 0x55, dtype=U8, device="cuda"), torch.full((5, sb + 4), 0x55, dtype=U8, device="cuda")
        eff.mx4_quantize(x, c[:, :cb], s[:, :sb])
        rc, rs = B.quantise(x.cpu())
        assert torch.equal(c[:, :cb].cpu(), B.pack(rc)) and torch.equal(s[:, :sb].cpu(), rs)
        assert (c[:, cb:] == 0x55).all() and (s[:, sb:] == 0x55).all()
        y = torch.full((5, 500), 5.0, dtype=BF, device="cuda")
        eff.mx4_dequantize(c[:, :cb], s[:, :sb], y[:, off:off + k])
        assert torch.equal(y[:, off:off + k].cpu().double(), B.values(B.pack(rc), rs)[:, :k])
        assert (y[:, :off] == 5).all() and (y[:, off + k:] == 5).all()
    row = big[:1, :256].expand(4, 256)                  # one row for all
    c, s = quantised(eff, row)
    assert (c == c[:1]).all() and (s == s[:1]).all()
    empty = torch.empty(0, 64, dtype=BF, device="cuda")
    quantised(eff, empty)
    eff.mx4_dequantize(*empty_rows(eff, 0, 64), empty)


def test_many_rows(eff):
    """More rows than one part of a launch, past 2^31 values."""
    m, k = (1 << 24) + 5, 136
    x = torch.empty(m, k, dtype=BF, device="cuda")
    x[:, ::2], x[:, 1::2] = 1.5, -0.25
    x[-1] = torch.linspace(-3, 3, k).to(BF).cuda()
    c, s = quantised(eff, x)
    for r in (0, 1 << 23, m - 1):
        rc, rs = B.quantise(x[r:r + 1].cpu())
        assert torch.equal(c[r:r + 1].cpu(), B.pack(rc)) and torch.equal(s[r:r + 1].cpu(), rs)
    assert (c[:-1] == c[0]).all() and (s[:-1] == s[0]).all()
    eff.mx4_dequantize(c, s, x)
    assert (x[:-1] == x[0]).all() and torch.equal(x[-1].cpu().double(), B.values(B.pack(rc), rs)[0, :k])
    del x, c, s
    torch.cuda.empty_cache()


# ---- products

def operands(eff, m, nw, k, dt, seed, groups=0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(m, k, generator=g) * torch.exp(torch.randn(m, 1, generator=g))).to(dt)
    w = (torch.randn(max(1, groups), nw, k, generator=g) * k ** -0.5).to(F32)
    wq, ws = quantised(eff, (w if groups else w[0]).cuda())
    return x, wq, ws


def check(eff, m, n, k, dt=BF, out=None, act=R.NONE, bias=False, residual=False, pre=False, groups=0, coded=False, seed=0, offsets=None):
    nw = 2 * n if act == R.SWIGLU else n
    x, wq, ws = operands(eff, m, nw, k, dt, seed + m + n + k, groups)
    g = torch.Generator().manual_seed(seed + 1)
    lead = (groups,) if groups else ()
    b = (torch.randn(*lead, nw, generator=g) * 0.5).to(dt) if bias else None
    res = torch.randn(m, n, generator=g).to(dt) if residual else None
    off = None
    if groups:
        if offsets is None:
            cuts = torch.sort(torch.randint(0, m + 1, (groups + 1,), generator=g))[0]
            cuts[0] = 0
            offsets = cuts.tolist()
        off = torch.tensor(offsets, dtype=I32)
    y = torch.full((m, n), 7.0, dtype=out or dt, device="cuda")
    p = torch.full((m, nw), 7.0, dtype=dt, device="cuda") if pre else None
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    xc, xs = quantised(eff, x.cuda())
    kw = dict(bias=cu(b), act=act, residual=cu(res), pre=p)
    args = (xc, wq, ws) if coded else (x.cuda(), wq, ws)
    if coded:
        kw["x_scales"] = xs
    if groups:
        eff.grouped_mx4_matmul(*args, off.cuda(), y, **kw)
    else:
        eff.mx4_matmul(*args, y, **kw)
    xv, wv = B.values(xc.cpu(), xs.cpu()), B.values(wq.cpu(), ws.cpu())
    ry, ye, rz, ze = R.matmul64(xv, wv, b, act, res, off, n)
    live = slice(0, m) if off is None else slice(int(off[0]), int(off[-1]))
    R.assert_within(y[live], ry[live], ye[live], "y")
    if p is not None:
        R.assert_within(p[live], rz[live], ze[live], "pre")
    for t in (y, p):
        if t is not None:
            assert (t[:live.start] == 7).all() and (t[live.stop:] == 7).all()
    return y


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 32, 33, 64, 100, 129, 300])
@pytest.mark.parametrize("n,k", [(1, 1), (8, 128), (20, 100), (64, 256), (65, 640), (130, 520), (515, 2563)])
def test_sizes(eff, m, n, k):
    check(eff, m, n, k, dt=BF if m % 2 else HF, coded=m % 3 == 0, bias=n > 20, residual=k > 300)


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("dt,out", [(BF, BF), (HF, HF), (BF, F32), (HF, F32)])
def test_epilogues(eff, act, dt, out):
    for m, n, k in ((5, 24, 384), (70, 96, 512), (150, 264, 320)):
        for bias, residual, pre in ((0, 0, 0), (1, 0, 1), (1, 1, 1), (0, 1, 0)):
            check(eff, m, n, k, dt, out, act, bool(bias), bool(residual), bool(pre), seed=act)


@pytest.mark.parametrize("m,n,k", [(257, 256, 1024), (512, 512, 512), (300, 520, 4096), (1025, 264, 2560), (2048, 1024, 640), (77, 4096, 256)])
def test_tiles(eff, m, n, k):
    check(eff, m, n, k, out=F32, coded=True)
    check(eff, m, n, k, act=R.SWIGLU, residual=True)


@pytest.mark.parametrize("groups,m", [(1, 40), (3, 0), (5, 5), (8, 150), (40, 64), (64, 700), (300, 200)])
def test_groups(eff, groups, m):
    for n, k, act in ((24, 130, R.SWIGLU), (72, 512, R.NONE)):
        check(eff, m, n, k, act=act, bias=True, pre=True, groups=groups)
        check(eff, m, n, k, dt=HF, act=act, groups=groups, coded=True, residual=True)


@pytest.mark.parametrize("path", PATHS, ids=lambda p: "-".join(map(str, p)))
def test_every_kernel(eff, path):
    """References on the GPU in float64: the sizes that reach the large tiles are large."""
    kind, m, n, k, act, groups = path
    nw = 2 * n if act == R.SWIGLU else n
    g = torch.Generator(device="cuda").manual_seed(m + n)
    x = torch.randn(m, k, generator=g, device="cuda", dtype=BF)
    wq, ws = quantised(eff, torch.randn(max(1, groups), nw, k, generator=g, device="cuda", dtype=BF) * k ** -0.5)
    off = None
    if groups:
        off = torch.tensor([0] + list(itertools.accumulate(group_sizes(m, groups))), dtype=I32, device="cuda")
    else:
        wq, ws = wq[0], ws[0]
    xc, xs = quantised(eff, x)
    b = torch.randn(*((groups,) if groups else ()), nw, generator=g, device="cuda").to(BF)
    res = torch.randn(m, n, generator=g, device="cuda").to(BF)
    for bias, residual, pre, out in ((None, None, False, BF), (None, res, False, BF), (b, res, True, F32)):
        y, p = torch.full((m, n), 7.0, dtype=out, device="cuda"), torch.full((m, nw), 7.0, dtype=BF, device="cuda") if pre else None
        kw = dict(x_scales=xs, bias=bias, residual=residual, pre=p, act=act)
        if groups:
            eff.grouped_mx4_matmul(xc, wq, ws, off, y, **kw)
        else:
            eff.mx4_matmul(xc, wq, ws, y, **kw)
        ry, ye, rz, ze = R.matmul64(B.values(xc, xs), B.values(wq, ws), bias, act, residual, off, n)
        R.assert_within(y, ry, ye, "y")
        if pre:
            R.assert_within(p, rz, ze, "pre")
    del ry, ye, rz, ze
    torch.cuda.empty_cache()


def test_groups_at_their_borders(eff):
    for off in ([0, 0, 0, 0], [0, 64, 64, 128], [0, 1, 65, 66], [0, 0, 0, 130], [0, 130, 130, 130], [3, 70, 71, 100], [0, 16, 32, 48]):
        check(eff, 130, 40, 256, groups=3, offsets=off, act=R.SWIGLU)


def test_offsets_from_elsewhere_are_clamped(eff):
    x, wq, ws = operands(eff, 20, 16, 128, BF, 1, 3)
    y = torch.zeros(20, 16, dtype=BF, device="cuda")
    for off in ([0, 10, 500, 900], [-5, 4, 4, 9], [30, 40, 50, 60], [0, 12, 6, 20]):
        eff.grouped_mx4_matmul(x.cuda(), wq, ws, torch.tensor(off, dtype=I32, device="cuda"), y)
    torch.cuda.synchronize()


def test_rows_in_no_group_are_not_read(eff):
    x, wq, ws = operands(eff, 90, 32, 256, BF, 1, 2)
    off = torch.tensor([0, 30, 61], dtype=I32, device="cuda")
    y, y2 = torch.zeros(90, 32, dtype=BF, device="cuda"), torch.zeros(90, 32, dtype=BF, device="cuda")
    eff.grouped_mx4_matmul(x.cuda(), wq, ws, off, y)
    x[61:] = NAN
    eff.grouped_mx4_matmul(x.cuda(), wq, ws, off, y2)
    assert torch.equal(y, y2) and not y[61:].any()


@pytest.mark.parametrize("m", [4, 40, 300])
def test_no_numbers_reach_their_rows_alone(eff, m):
    x, wq, ws = operands(eff, m, 48, 640, BF, 2)
    x[1, 3], x[m - 1, 639] = INF, NAN
    y = torch.zeros(m, 48, dtype=BF, device="cuda")
    eff.mx4_matmul(x.cuda(), wq, ws, y)
    assert torch.isnan(y[[1, m - 1]]).all() and torch.isfinite(y[[i for i in range(m) if i not in (1, m - 1)]]).all()
    ws[5, 7] = 255
    y.zero_()
    x[1, 3], x[m - 1, 639] = 1.0, 1.0
    eff.mx4_matmul(x.cuda(), wq, ws, y)
    assert torch.isnan(y[:, 5]).all() and torch.isfinite(y[:, [i for i in range(48) if i != 5]]).all()


def test_large_and_small_scales(eff):
    """Products whose scales are far from one, within the normal numbers of fp32."""
    for e in (-50, 0, 55):
        x, wq, ws = operands(eff, 20, 24, 256, BF, 3)
        x = torch.ldexp(x.float(), torch.tensor(e)).to(BF)
        xc, xs = quantised(eff, x.cuda())
        ws2 = (ws.int() + (e if e < 0 else 0)).clamp(0, 254).to(U8)
        y = torch.zeros(20, 24, dtype=F32, device="cuda")
        eff.mx4_matmul(xc, wq, ws2, y, x_scales=xs)
        xv, wv = B.values(xc.cpu(), xs.cpu()), B.values(wq.cpu(), ws2.cpu())
        ry, ye, _, _ = R.matmul64(xv, wv, None, R.NONE, None, None, 24)
        R.assert_within(y, ry, ye, "y")


def test_operand_strides(eff):
    """Rows of codes and scales apart, one row for all, and groups apart."""
    m, n, k = 70, 40, 384
    x, wq, ws = operands(eff, m, n, k, BF, 5)
    xc, xs = quantised(eff, x.cuda())
    want = torch.empty(m, n, dtype=BF, device="cuda")
    eff.mx4_matmul(xc, wq, ws, want, x_scales=xs)
    wide = lambda t, a: torch.cat([t, torch.full((t.shape[0], a), 0x77, dtype=U8, device="cuda")], 1)[:, :t.shape[1]]  # noqa: E731
    y = torch.full((m, n + 9), 7.0, dtype=BF, device="cuda")
    eff.mx4_matmul(wide(xc, 16), wide(wq, 48), wide(ws, 8), y[:, :n], x_scales=wide(xs, 4))
    assert torch.equal(y[:, :n], want) and (y[:, n:] == 7).all()
    big = torch.randn(2 * m, k + 40).to(BF).cuda()
    xv = big[::2, 1:k + 1]                              # 16-bit rows at an odd place
    y2, y3 = torch.empty(m, n, dtype=BF, device="cuda"), torch.empty(m, n, dtype=BF, device="cuda")
    eff.mx4_matmul(xv, wq, ws, y2)
    eff.mx4_matmul(xv.contiguous(), wq, ws, y3)
    assert torch.equal(y2, y3)
    one = torch.empty(m, n, dtype=BF, device="cuda")
    eff.mx4_matmul(xc[:1].expand(m, -1), wq, ws, one, x_scales=xs[:1].expand(m, -1))
    assert torch.equal(one, want[:1].expand(m, n))
    w3, s3 = torch.stack([wq, wq]), torch.stack([ws, ws])
    off = torch.tensor([0, 30, 70], dtype=I32, device="cuda")
    eff.grouped_mx4_matmul(xc, wq[None].expand(2, -1, -1), ws[None].expand(2, -1, -1), off, y2, x_scales=xs)
    eff.grouped_mx4_matmul(xc, w3, s3, off, y3, x_scales=xs)
    assert torch.equal(y2, y3)
    torch.testing.assert_close(y2.float(), want.float(), rtol=2 ** -7, atol=1e-3)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("m,n,k,act", [(1, 40, 8, 0), (3, 72, 136, 4), (16, 64, 1000, 0), (9, 520, 2560, 4), (13, 40, 264, 4), (5, 24, 520, 0),
                                     (40, 264, 520, 0), (250, 40, 1032, 4), (129, 130, 2568, 0)])
def test_16_bit_rows_quantised_inside(eff, m, n, k, act, dt):
    """Few rows: the kernel quantises x itself, at any place and row distance, k inside a block, a unit and a chunk of two: the bits
    of quantising first.  What lies beside the rows may hold anything."""
    nw = 2 * n if act == R.SWIGLU else n
    x, wq, ws = operands(eff, m, nw, k, dt, m + k)
    if k >= 264:
        x[0, 100], x[m - 1, 5] = 0.0, 3e4
        x[m // 2, 64:96] = 0
    want = torch.empty(m, n, dtype=dt, device="cuda")
    xc, xs = quantised(eff, x.cuda())
    eff.mx4_matmul(xc, wq, ws, want, x_scales=xs, act=act)
    for off, pad in ((0, 0), (1, 5), (3, 13)):
        big = torch.full((m, k + off + pad), NAN, dtype=dt, device="cuda")
        big[:, off:off + k] = x.cuda()
        y = torch.empty_like(want)
        eff.mx4_matmul(big[:, off:off + k], wq, ws, y, act=act)
        assert torch.equal(y, want), (off, pad)
    g3 = torch.empty(m, n, dtype=dt, device="cuda")
    eff.grouped_mx4_matmul(x.cuda(), wq[None], ws[None], torch.tensor([0, m], dtype=I32, device="cuda"), g3, act=act)
    assert torch.equal(g3, want)
    x[m - 1, k - 1] = INF
    eff.mx4_matmul(x.cuda(), wq, ws, g3, act=act)
    assert torch.isnan(g3[m - 1]).all() and torch.equal(g3[:m - 1], want[:m - 1])


def test_one_very_wide_16_bit_row_for_all(eff):
    """x and W one row each, broadcast: -1, 0 and 1 are whole numbers in 4 bits, and so are the sums below 2^24 in fp32, in any order."""
    m, n, k = ONE_ROW_WIDE
    g = torch.Generator().manual_seed(3)
    x, w = (torch.randint(-1, 2, (1, k), generator=g, dtype=torch.int8) for _ in range(2))
    want = int((x.int() * w.int()).sum())
    assert 0 < abs(want) < 1 << 24 and int((x & 1).sum()) > 1 << 24
    xc = x.cuda().to(BF)
    wq, ws = quantised(eff, w.cuda().to(BF))
    y = torch.empty(m, n, dtype=F32, device="cuda")
    eff.mx4_matmul(xc.expand(m, -1), wq.expand(n, -1), ws.expand(n, -1), y)
    assert (y == want).all()
    del x, w, xc, wq, ws, y
    torch.cuda.empty_cache()


def test_residual_in_place_and_no_rows(eff):
    x, wq, ws = operands(eff, 33, 64, 128, BF, 7)
    r = torch.randn(33, 64).to(BF).cuda()
    y = torch.empty_like(r)
    eff.mx4_matmul(x.cuda(), wq, ws, y, residual=r)
    eff.mx4_matmul(x.cuda(), wq, ws, r, residual=r)
    assert torch.equal(y, r)
    eff.mx4_matmul(torch.empty(0, 128, dtype=BF, device="cuda"), wq, ws, torch.empty(0, 64, dtype=BF, device="cuda"))


@pytest.mark.parametrize("m,n,k,act", [(1, 512, 2560, R.GELU), (16, 2048, 4096, R.SWIGLU), (4096, 1024, 4096, R.NONE)])
def test_full_sizes(eff, m, n, k, act):
    check(eff, m, n, k, act=act, out=F32)
