"""Groups of 4-bit products whose offsets lie outside the rows: what is inside is right, what is in no group and what lies around the
operands stays, in every kernel, with x in codes and in 16 bits."""
import itertools

import pytest
import torch

from tests import block_ref as B
from tests import ops_ref as R
from tests.matmul_paths import group_sizes
from tests.mx4_paths import PATHS
from tests.test_gpu_mx4 import quantised

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
NAN = float("nan")
AROUND = 32           # rows before and behind


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    return e


def inside(t, fill):
    """t between rows of `fill`: the whole, and t's place in it."""
    whole = torch.full((t.shape[0] + 2 * AROUND, t.shape[1]), fill, dtype=t.dtype, device="cuda")
    part = whole[AROUND:AROUND + t.shape[0]]
    part.copy_(t)
    return whole, part


class Case:
    def __init__(self, eff, path):
        _, self.m, self.n, k, self.act, self.groups = path
        self.eff, self.nw = eff, 2 * self.n if self.act == R.SWIGLU else self.n
        g = torch.Generator(device="cuda").manual_seed(self.m + self.n)
        x = torch.randn(self.m, k, generator=g, device="cuda", dtype=BF)
        self.w = quantised(eff, torch.randn(self.groups, self.nw, k, generator=g, device="cuda", dtype=BF) * k ** -0.5)
        codes, scales = quantised(eff, x)
        self.x, self.codes, self.scales = inside(x, NAN)[1], inside(codes, 0x77)[1], inside(scales, 255)[1]   # around: NaN
        self.off = [0] + list(itertools.accumulate(group_sizes(self.m, self.groups)))

    def run(self, off, coded):
        """y and pre among rows of 7."""
        (yw, y), (pw, p) = [inside(torch.full((self.m, c), 7.0, dtype=BF, device="cuda"), 7.0) for c in (self.n, self.nw)]
        off = torch.tensor(off, dtype=I32, device="cuda")
        kw = dict(x_scales=self.scales) if coded else {}
        self.eff.grouped_mx4_matmul(self.codes if coded else self.x, *self.w, off, y, act=self.act, pre=p, **kw)
        plain_w, plain = inside(torch.full((self.m, self.n), 7.0, dtype=BF, device="cuda"), 7.0)     # without pre: the other way out
        self.eff.grouped_mx4_matmul(self.codes if coded else self.x, *self.w, off, plain, act=self.act, **kw)
        for t in (yw, pw, plain_w):
            assert (t[:AROUND] == 7).all() and (t[-AROUND:] == 7).all(), "written around the rows"
        return y, p, plain


@pytest.mark.parametrize("path", [p for p in PATHS if p[5]], ids=lambda p: "-".join(map(str, p)))
def test_offsets_outside_the_rows(eff, path):
    c = Case(eff, path)
    m, third = c.m, c.m // 3
    far = list(c.off)
    far[0], far[-1] = -2 ** 31, 2 ** 31 - 1
    xv, wv = B.values(c.codes, c.scales), B.values(*c.w)
    for off in ([o - third for o in c.off], [o + third for o in c.off], [o + 2 * m for o in c.off], [o - 2 * m for o in c.off], far):
        clamped = torch.tensor(off).clamp(0, m)
        ry, ye, rz, ze = R.matmul64(xv, wv, None, c.act, None, clamped, c.n)
        live = slice(int(clamped[0]), int(clamped[-1]))
        for coded in (True, False):
            y, p, plain = c.run(off, coded)
            R.assert_within(y[live], ry[live], ye[live], "y")
            R.assert_within(plain[live], ry[live], ye[live], "y without pre")
            R.assert_within(p[live], rz[live], ze[live], "pre")
            for t in (y, p, plain):
                assert (t[:live.start] == 7).all() and (t[live.stop:] == 7).all(), "rows in no group"
    del xv, wv, ry, ye, rz, ze
    torch.cuda.empty_cache()


@pytest.mark.parametrize("path", [p for p in PATHS if p[5]], ids=lambda p: "-".join(map(str, p)))
def test_offsets_that_do_not_ascend(eff, path):
    """Not what a caller may pass, and nothing is said of y, but nothing beside the outputs is written."""
    c = Case(eff, path)
    swapped = list(c.off)
    swapped[1], swapped[-2] = swapped[-2], swapped[1]
    for off in (c.off[::-1], swapped, [c.m, -5] + c.off[2:]):
        for coded in (True, False):
            c.run(off, coded)
