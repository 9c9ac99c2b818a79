"""Sizes that the operators without an engine refuse before anything is launched (no GPU needed)."""
import pytest

from tests.test_ops_refusals import A, backward, desc, eff  # noqa: F401


@pytest.mark.parametrize("kw,out", [(dict(n=1 << 22, k=1 << 16), "dw"), (dict(n=1 << 22, k=1 << 16, groups=8, stride_dw=1 << 38), "dw"),
                                    (dict(n=1 << 30, k=8), "dbias"), (dict(n=1 << 29, k=8, act=4), "dbias")])
def test_gradients_of_no_rows_that_no_grid_holds(eff, kw, out):  # noqa: F811
    """m = 0 writes zeros to dw and dbias, with the same bound on their size as any other m."""
    ld = kw["k"]
    kw = dict(m=0, ld_x=ld, ld_w=ld, ld_dx=ld, ld_dw=ld, ld_y=kw["n"], ld_pre=2 * kw["n"], stride_w=kw.get("stride_dw", 0), **kw)
    want = dict(dx=None, dw=A if out == "dw" else None, dbias=A if out == "dbias" else None)
    assert backward(eff, desc(**kw), offsets=A if kw.get("groups") else None, **want) == eff.EFF_EINVAL
