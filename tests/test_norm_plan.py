"""How many rows and columns one launch of layer norm takes, asked of the library without a GPU."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    import expert_ffn_serving_amd as eff
    hipcc = "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    eff.lib()
    lib = os.path.join(ROOT, "expert_ffn_serving_amd")
    so = str(tmp_path_factory.mktemp("shim") / "libnormshim.so")
    subprocess.check_call([hipcc, "-O2", "-std=c++17", "--offload-arch=gfx950", "--cuda-host-only", "-fPIC", "-shared", "-o", so,
                           os.path.join(ROOT, "tests", "native", "norm_plan_shim.cpp"), "-L" + lib, "-l:libeff.so", "-Wl,-rpath," + lib])
    return ctypes.CDLL(so)


@pytest.mark.parametrize("threads,per", [(256, 4), (512, 4), (512, 2), (1024, 2), (1024, 1)])    # every workgroup of the row kernels
def test_a_launchs_threads_stay_below_2_32(shim, threads, per):
    """A launch of 2^32 threads or more is refused by the runtime: rows are split before, as late as that allows."""
    f = shim.shim_norm_at_once
    f.restype, f.argtypes = ctypes.c_int64, [ctypes.c_int, ctypes.c_int64]
    rows = f(threads, per)
    assert rows % per == 0
    assert rows // per * threads < 1 << 32 <= (rows // per + 1) * threads


def test_the_columns_of_a_launch_too(shim):
    """64 columns to a workgroup of 1024 threads, which add up the partial sums of dw and db."""
    shim.shim_norm_columns_at_once.restype = ctypes.c_int64
    cols = shim.shim_norm_columns_at_once()
    assert cols % 64 == 0 and cols // 64 * 1024 < 1 << 32
