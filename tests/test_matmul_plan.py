"""Which kernel a product takes, asked of the library without a GPU: what a tile's kernel can address is what it is given."""
import ctypes
import itertools
import os
import random
import subprocess

import pytest

from expert_ffn_serving_amd.ops import MatmulDesc
from tests.matmul_paths import PATHS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ANY, FEW1, FEW2, BIG, WIDE, MID, LOW = range(7)
TILES = {BIG: (256, 256, 64), WIDE: (128, 256, 32), MID: (128, 128, 64), LOW: (64, 128, 64)}   # rows, columns, k of a step
FORWARD, DX, DW = range(3)


def library():
    import expert_ffn_serving_amd as eff
    eff.lib()
    return os.path.join(ROOT, "expert_ffn_serving_amd", "libeff.so")


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    hipcc = "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    lib = library()
    so = str(tmp_path_factory.mktemp("shim") / "libplanshim.so")
    subprocess.check_call([hipcc, "-O2", "-std=c++17", "--offload-arch=gfx950", "--cuda-host-only", "-fPIC", "-shared", "-o", so,
                           os.path.join(ROOT, "tests", "native", "matmul_plan_shim.cpp"),
                           "-L" + os.path.dirname(lib), "-l:libeff.so", "-Wl,-rpath," + os.path.dirname(lib)])
    shim = ctypes.CDLL(so)

    def ask(m, n, k, product=FORWARD, act=0, groups=0, pad=0, ld=None, dtype=0, out=None):
        """kind, parts of k, elements between the rows of x and of w, as read."""
        nw = 2 * n if act == 4 else n
        d = MatmulDesc(dtype, dtype if out is None else out, act, groups, m, n, k, *((ld or k + pad),) * 2, n + pad, n + pad, nw + pad,
                       nw * (ld or k + pad), k + pad, k + pad, nw * (k + pad))
        res = (ctypes.c_int64 * 4)()
        shim.shim_matmul_choice(ctypes.byref(d), product, res)
        return tuple(res)
    return ask


def reach(m, n, k, product, act, kind, ld_x, ld_w):
    """The largest byte offset from a tile's first element that its kernel computes in 32 bits, for x and for w."""
    bm, bn, bk = TILES[kind]
    nw = 2 * n if act == 4 else n
    M, N = ((m, n), (m, k), (nw, k))[product]        # rows and columns of the product's output
    cols = min(bn // 2 if act == 4 and product == FORWARD else bn, N)
    x = ((min(bm, M) - 1) * ld_x + bk if product != DW else (bk - 1) * ld_x + bm) * 2
    w = ((cols - 1) * ld_w + bk if product == FORWARD else (bk - 1) * ld_w + bn) * 2
    return x, w


LONG = [(64, 128, 17825792, FORWARD, 0), (1024, 1024, 8650752, FORWARD, 0), (1024, 1024, (1 << 31) - 1, FORWARD, 0),
        (300, 40, 1 << 24, FORWARD, 4), (33, 1, 1 << 26, FORWARD, 0), (1024, 1 << 24, 8, DX, 0), (64, 1 << 26, 8, DW, 1),
        (4096, 8, 1 << 26, DW, 0)]


@pytest.mark.parametrize("m,n,k,product,act", LONG)
def test_long_rows_stay_within_32_bit_offsets(choice, m, n, k, product, act):
    kind, _, ld_x, ld_w = choice(m, n, k, product, act)
    if kind in TILES:
        assert max(reach(m, n, k, product, act, kind, ld_x, ld_w)) < 1 << 32, (kind, ld_x, ld_w)


def test_any_rows_stay_within_32_bit_offsets(choice):
    rng = random.Random(1)
    taken = {}
    for _ in range(20000):
        m, n, k = (int(2 ** rng.uniform(0, top)) for top in (20, 30, 31))
        product, act = rng.choice([FORWARD, DX, DW]), rng.choice([0, 1, 4])
        pad = rng.choice([0, 0, 1, 8])
        if product == DX and m * n > 1 << 40:
            continue
        kind, _, ld_x, ld_w = choice(m, n, k, product, act, pad=pad)
        taken[kind] = taken.get(kind, 0) + 1
        if kind in TILES:
            assert max(reach(m, n, k, product, act, kind, ld_x, ld_w)) < 1 << 32, (m, n, k, product, act, pad, kind)
    assert set(taken) == set(range(7))


def test_rows_that_fit_keep_their_tiles(choice):
    """The tiles are given up only for rows that they cannot address."""
    assert choice(256, 256, (1 << 23) - 8)[0] in TILES and choice(64, 128, (1 << 24) - 64)[0] in TILES
    assert choice(1, 8, (1 << 31) - 1)[0] == FEW1        # W streamed through registers: addresses of 64 bits


def test_the_paths_reach_every_tile(choice):
    reached = set()
    for product, m, n, k, act, groups in PATHS:
        for dtype in (0, 1):
            kind, splits = choice(m, n, k, product, act, groups, dtype=dtype)[:2]
            reached.add((product, groups > 0, act == 4 and product == FORWARD, kind, splits > 1, dtype))
    want = set()
    for product, grouped, glu, kind, split, dtype in itertools.product((FORWARD, DX, DW), (False, True), (False, True), range(FEW1, LOW + 1),
                                                                       (False, True), (0, 1)):
        if split and (grouped or kind in (FEW1, FEW2)):     # k is split where there is one product of few tiles
            continue
        if product != FORWARD and (glu or kind in (FEW1, FEW2)):
            continue
        want.add((product, grouped, glu, kind, split, dtype))
    assert reached == want
