"""Which kernel a product of 4-bit operands takes, asked of the library without a GPU."""
import ctypes
import os
import random
import subprocess

import pytest

from expert_ffn_serving_amd.ops import Mx4Desc, mx4_row_bytes
from tests.mx4_paths import BIG, FEW1, FEW2, FEW4, LOW, MID, ONE_ROW_WIDE, PATHS, THIN

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TILE_ROWS = {BIG: 256, MID: 128, LOW: 128, THIN: 128}     # the larger side of a tile


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    import expert_ffn_serving_amd as eff
    hipcc = "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    eff.lib()
    lib = os.path.join(ROOT, "expert_ffn_serving_amd")
    so = str(tmp_path_factory.mktemp("shim") / "libmx4shim.so")
    subprocess.check_call([hipcc, "-O2", "-std=c++17", "--offload-arch=gfx950", "--cuda-host-only", "-fPIC", "-shared", "-o", so,
                           os.path.join(ROOT, "tests", "native", "mx4_plan_shim.cpp"), "-L" + lib, "-l:libeff.so", "-Wl,-rpath," + lib])
    shim = ctypes.CDLL(so)

    def ask(m, n, k, act=0, groups=0, ld=None):
        nw = 2 * n if act == 4 else n
        cb, sb = mx4_row_bytes(k)
        ld = ld or cb
        return shim.shim_mx4_choice(ctypes.byref(Mx4Desc(3, 0, 0, act, groups, 0, m, n, k, ld, sb, ld, sb, nw * ld, nw * sb, n, n, nw)))
    return ask


def test_the_paths_take_the_kernels_they_are_for(choice):
    for kind, m, n, k, act, groups in PATHS:
        assert choice(m, n, k, act, groups) == kind, (kind, m, n, k, act, groups)
    assert {p[0] for p in PATHS} == {FEW1, FEW2, FEW4, BIG, MID, LOW, THIN}


def test_what_a_tiles_offsets_reach(choice):
    """A tile's lanes hold 32-bit byte offsets from its first row: rows further apart take the kernels that stream W, or a tile of
    fewer rows."""
    rng = random.Random(1)
    for _ in range(4000):
        m, n, k = rng.randint(1, 20000), rng.randint(1, 9000), rng.randint(1, 9000)
        ld = max(mx4_row_bytes(k)[0], 16 * rng.randint(1, 1 << rng.randint(1, 30)))
        kind = choice(m, n, k, rng.choice([0, 4]), rng.choice([0, 0, 3, 100]), ld)
        if kind in TILE_ROWS:
            assert TILE_ROWS[kind] * ld < 1 << 32
    assert choice(8192, 4096, 4096) == BIG and choice(8192, 4096, 4096, ld=1 << 24) == MID and choice(8192, 4096, 4096, ld=1 << 25) == FEW4
    assert choice(8192, 4096, 4096, ld=1 << 58) == FEW4    # whose product with a tile's rows passes 64 bits


def test_16_bit_rows_are_planned_once(choice):
    """Distances of x decide with whether a tile can be taken.  16-bit rows that the kernel quantises itself have other ones than
    their codes would: a case where the two would choose differently, which tests/test_gpu_mx4.py runs."""
    m, n, k = ONE_ROW_WIDE
    cb, _ = mx4_row_bytes(k)
    assert choice(m, n, k, ld=cb) == FEW1 and choice(m, n, k, ld=16) in TILE_ROWS
