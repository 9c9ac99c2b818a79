"""Products over rows of many millions of values: addresses past 32 bits inside one tile, and k up to the largest.  The
operands hold small whole numbers in a few columns and zeros elsewhere, so that every sum is exact in fp32."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    yield e
    torch.cuda.empty_cache()


def columns(k, count, seed):
    """Columns of a long row: both ends, the middle, and others anywhere."""
    g = torch.Generator().manual_seed(seed)
    at = torch.cat([torch.randint(0, k, (count,), generator=g), torch.tensor([0, 1, k - 1, k - 2, k // 2])])
    return at.unique()


def sparse(rows, k, at, seed):
    """[rows, k] of zeros with whole numbers of at most 2 in the columns `at`, and those columns in 64 bits."""
    v = torch.randint(-2, 3, (rows, len(at)), generator=torch.Generator().manual_seed(seed)).double().cuda()
    t = torch.zeros((rows, k), dtype=BF, device="cuda")
    t[:, at.cuda()] = v.to(BF)
    return t, v


# 64 x 128 tiles whose offsets pass 2^31; rows that no tile can address; W streamed with the largest k, whole vectors or not
@pytest.mark.parametrize("m,n,k", [(64, 128, 12 << 20), (64, 128, 17825792), (40, 130, (12 << 20) + 5), (1, 2, (1 << 31) - 8),
                                   (1, 1, (1 << 31) - 1), (17, 3, (1 << 24) + 3)])
def test_long_k(eff, m, n, k):
    at = columns(k, 300, m)
    x, xv = sparse(m, k, at, 1)
    w, wv = sparse(n, k, at, 2)
    y = torch.full((m, n), 7.0, dtype=F32, device="cuda")
    eff.matmul(x, w, y)
    assert torch.equal(y.double(), xv @ wv.t()), (m, n, k)
    del x, w
    torch.cuda.empty_cache()


def test_gradients_of_many_columns(eff):
    """dy of 64 rows of 34 million columns: both of its products would pass 2^32 bytes inside a tile."""
    m, n, k = 64, 34 * (1 << 20), 8
    at = columns(n, 60, 3)
    dy, dv = sparse(m, n, at, 4)
    w = torch.randint(-2, 3, (n, k), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda", dtype=torch.int8).to(BF)
    x = torch.randint(-2, 3, (m, k), generator=torch.Generator().manual_seed(6)).to(BF).cuda()
    dx, dw = torch.full((m, k), 7.0, dtype=BF, device="cuda"), torch.full((n, k), 7.0, dtype=BF, device="cuda")
    eff.matmul_backward(dy, x, w, dx=dx, dw=dw)
    at = at.cuda()
    assert torch.equal(dx, (dv @ w[at].double()).to(BF))
    assert torch.equal(dw[at], (dv.t() @ x.double()).to(BF))
    dw[at] = 0
    assert not dw.any()
    del dy, w, dw
    torch.cuda.empty_cache()
