"""Sizes and overlaps that the operators without an engine refuse before anything is launched (no GPU needed)."""
import pytest

from tests.test_ops_refusals import A, backward, desc, eff, forward  # noqa: F401


@pytest.mark.parametrize("kw,out", [(dict(n=1 << 22, k=1 << 16), "dw"), (dict(n=1 << 22, k=1 << 16, groups=8, stride_dw=1 << 38), "dw"),
                                    (dict(n=1 << 30, k=8), "dbias"), (dict(n=1 << 29, k=8, act=4), "dbias")])
def test_gradients_of_no_rows_that_no_grid_holds(eff, kw, out):  # noqa: F811
    """m = 0 writes zeros to dw and dbias, with the same bound on their size as any other m."""
    ld = kw["k"]
    kw = dict(m=0, ld_x=ld, ld_w=ld, ld_dx=ld, ld_dw=ld, ld_y=kw["n"], ld_pre=2 * kw["n"], stride_w=kw.get("stride_dw", 0), **kw)
    want = dict(dx=None, dw=A if out == "dw" else None, dbias=A if out == "dbias" else None)
    assert backward(eff, desc(**kw), offsets=A if kw.get("groups") else None, **want) == eff.EFF_EINVAL


@pytest.mark.parametrize("kw", [dict(ld_residual=0), dict(ld_residual=16), dict(out_dtype=2), dict(out_dtype=2, m=1)])
def test_residual_in_place_of_another_layout(eff, kw):  # noqa: F811
    """y may be the residual itself: the same elements of the same size.  A row of y that is added to every row, rows at another
    distance or 16-bit values under fp32 ones would be overwritten before they are read."""
    assert forward(eff, desc(**kw), residual=A, y=A) == eff.EFF_EINVAL


@pytest.mark.parametrize("ld", [0, 16])
def test_combined_in_place_of_another_layout(eff, ld):  # noqa: F811
    assert eff.lib().eff_combine_tokens(0, A << 4, 8, 8, A << 5, A << 6, 4, 2, 8, A, ld, A, 8, None) == eff.EFF_EINVAL
