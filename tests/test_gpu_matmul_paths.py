"""Every tile of the products' kernel in every layout of its operands, whole and with k split, dense and in groups of which one
is empty, against 64 bits (sizes: matmul_paths)."""
import pytest
import torch

from tests import ops_ref as R
from tests.matmul_paths import FORWARD, DX, PATHS, group_sizes
from tests.test_gpu_matmul import run_backward, run_forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    return e


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("product,m,n,k,act,groups", PATHS)
def test_path(eff, product, m, n, k, act, groups, dtype):
    counts = group_sizes(m, groups) if groups else None
    if product == FORWARD:
        run_forward(eff, m, n, k, dtype=dtype, act=act, counts=counts)
        run_forward(eff, m, n, k, dtype=dtype, act=act, counts=counts, bias=True, residual=True, pre=True)
        run_forward(eff, m, n, k, dtype=dtype, act=act or R.GELU, counts=counts, residual=True, out=torch.float32)
    else:
        run_backward(eff, m, n, k, dtype=dtype, act=act, counts=counts, want=("dx",) if product == DX else ("dw",))


def shifted(t, by):
    """The same values in memory that begins `by` elements behind a multiple of 16 bytes."""
    buf = torch.zeros(t.numel() + 16, dtype=t.dtype, device="cuda")
    v = buf[by:by + t.numel()].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("which", ["x", "w", "dy", "all"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("m,n,k,groups", [(300, 264, 520, 0), (1030, 520, 264, 0), (20, 72, 136, 0), (517, 136, 264, 5)])
def test_pointers_that_are_not_aligned(eff, m, n, k, groups, dtype, which):
    """Forward and gradients at tile sizes with operands and outputs that begin anywhere.  Whole numbers up to 2: the sums are
    exact in fp32 and rounded once."""
    g = torch.Generator().manual_seed(m)
    whole = lambda *s: torch.randint(-2, 3, s, generator=g).to(dtype)  # noqa: E731
    counts = group_sizes(m, groups) if groups else None
    lead = (groups,) if groups else ()
    x, w, dy = whole(m, k), whole(*lead, n, k), whole(m, n)
    put = {name: shifted(t, 3) if which in (name, "all") else t.cuda() for name, t in (("x", x), ("w", w), ("dy", dy))}
    y, dx, dw = (shifted(torch.zeros(s, dtype=dtype), 5 if which == "all" else 0) for s in ((m, n), (m, k), (*lead, n, k)))
    if counts:
        off = torch.tensor([sum(counts[:i]) for i in range(groups + 1)], dtype=torch.int32)
        eff.grouped_matmul(put["x"], put["w"], off.cuda(), y)
        eff.grouped_matmul_backward(put["dy"], put["x"], put["w"], off.cuda(), dx=dx, dw=dw)
    else:
        off = None
        eff.matmul(put["x"], put["w"], y)
        eff.matmul_backward(put["dy"], put["x"], put["w"], dx=dx, dw=dw)
    for e, rows in R.groups_of(off, m):
        xr, dr, we = x[rows].double(), dy[rows].double(), (w if e is None else w[e]).double()
        assert torch.equal(y[rows].cpu(), (xr @ we.t()).to(dtype))
        assert torch.equal(dx[rows].cpu(), (dr @ we).to(dtype))
        assert torch.equal((dw if e is None else dw[e]).cpu(), (dr.t() @ xr).to(dtype))
