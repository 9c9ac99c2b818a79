"""The router's losses, the experts' counts and the gradient at the logits against 64 bits (tests/block_ref.py)."""
import math

import pytest
import torch

from tests import block_ref as B
from tests import ops_ref as R

pytestmark = pytest.mark.gpu
BF, HF, F32, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    return e


def batch(T, E, K, dt, seed, unrouted=0.1):
    g = torch.Generator().manual_seed(seed)
    logits = (torch.randn(T, E, generator=g) * 2 + torch.randn(E, generator=g)).to(dt)
    ids = torch.topk(logits.float(), K, dim=1)[1].to(I32)
    ids[torch.rand(T, K, generator=g) < unrouted] = -1
    w = torch.softmax(torch.randn(T, K, generator=g), 1)
    dw = torch.randn(T, K, generator=g)
    return logits, ids.contiguous(), w, dw


def forward(eff, logits, ids, mask=None):
    T, E = logits.shape
    counts = torch.full((E + 1,), -7, dtype=I32, device="cuda")
    lse, losses = torch.full((T,), NAN, device="cuda"), torch.full((2,), NAN, device="cuda")
    eff.balance_loss(logits.cuda() if not logits.is_cuda else logits, ids.cuda(), counts, lse, losses, mask=None if mask is None else mask.cuda())
    return counts, lse, losses


def check(eff, logits, ids, mask=None):
    counts, lse, losses = forward(eff, logits, ids, mask)
    rl, le, rc, rs, se = B.balance64(logits, ids, mask, logits.shape[1])
    assert torch.equal(counts.cpu().long(), rc)
    dead = rs == -math.inf
    assert torch.equal(lse.cpu() == -math.inf, dead)
    R.assert_within(lse[~dead.cuda()], rs[~dead], se[~dead], "lse")
    past = rl > torch.finfo(F32).max                   # no fp32 number is as large: infinite
    assert (losses.cpu()[past] == INF).all()
    R.assert_within(losses[~past.cuda()], rl[~past], le[~past], "losses")
    return counts, lse, losses


def check_grad(eff, logits, ids, counts, lse, dlosses, w, dw):
    out = torch.full(logits.shape, NAN, dtype=logits.dtype, device="cuda")
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    eff.balance_loss_backward(logits.cuda(), ids.cuda(), counts, lse, cu(dlosses), out, w=cu(w), dw=cu(dw))
    ref, err = B.balance_grad64(logits, ids, counts.cpu().long(), lse.cpu(), dlosses, w, dw)
    R.assert_within(out, ref, err, "dlogits")
    return out


@pytest.mark.parametrize("E", [1, 2, 3, 4, 8, 60, 64, 65, 160, 256, 257, 512, 520, 1000, 1024, 1032, 2048, 2050, 4096])
@pytest.mark.parametrize("dt", [F32, BF, HF])
def test_experts(eff, E, dt):
    for T, K in ((1, 1), (70, min(E, 6))):
        logits, ids, w, dw = batch(T, E, K, dt, E + T)
        counts, lse, _ = check(eff, logits, ids)
        check_grad(eff, logits, ids, counts, lse, torch.tensor([0.7, -0.2]), w, dw)


@pytest.mark.parametrize("T", [2, 8, 9, 64, 1000, 2049, 5000])
def test_tokens(eff, T):
    logits, ids, w, dw = batch(T, 40, 4, F32, T)
    g = torch.Generator().manual_seed(T)
    mask = torch.rand(T, generator=g) > 0.3
    counts, lse, _ = check(eff, logits, ids, mask)
    check_grad(eff, logits, ids, counts, lse, torch.tensor([1e-2, 1e-3]), w, dw)


@pytest.mark.parametrize("T,E", [(16, 1100), (17, 1100), (63, 40), (64, 1024), (65, 40), (66, 1024)])
def test_few_tokens(eff, T, E):
    """About where one workgroup no longer takes all of them."""
    logits, ids, _, _ = batch(T, E, 4, BF, T + E)
    check(eff, logits, ids, torch.arange(T) % 5 != 3)


def test_parts_of_the_gradient(eff):
    logits, ids, w, dw = batch(33, 24, 3, F32, 5)
    counts, lse, _ = check(eff, logits, ids)
    one = check_grad(eff, logits, ids, counts, lse, torch.tensor([1.0, 0.0]), None, None)
    two = check_grad(eff, logits, ids, counts, lse, torch.tensor([0.0, 1.0]), None, None)
    three = check_grad(eff, logits, ids, counts, lse, None, w, dw)
    every = check_grad(eff, logits, ids, counts, lse, torch.tensor([1.0, 1.0]), w, dw)
    torch.testing.assert_close(one + two + three, every, rtol=1e-5, atol=1e-6)
    assert one.abs().sum() > 0 and two.abs().sum() > 0 and three.abs().sum() > 0


def test_all_top_k(eff):
    for K in (1, 2, 31, 32):
        logits, ids, w, dw = batch(50, 48, K, F32, K)
        counts, lse, _ = check(eff, logits, ids)
        check_grad(eff, logits, ids, counts, lse, torch.tensor([1.0, 1.0]), w, dw)


def test_the_same_expert_twice_and_ids_outside(eff):
    logits, ids, w, dw = batch(40, 16, 5, F32, 3, 0.0)
    ids[:, 1] = ids[:, 0]
    ids[::3, 4] = ids[::3, 0]
    ids[::4, 2], ids[1::4, 2], ids[2::4, 2] = 16, -5, 2 ** 31 - 1
    w[::4, 2] = dw[1::4, 2] = NAN                     # of an unrouted pair: not used
    counts, lse, _ = check(eff, logits, ids)
    check_grad(eff, logits, ids, counts, lse, torch.tensor([0.5, 0.1]), w, dw)


def test_masked_tokens_and_logits(eff):
    """Padding holds anything; rows and experts at -infinity; lowest finite values; no token left at all."""
    logits, ids, w, dw = batch(64, 32, 4, F32, 8)
    mask = torch.ones(64, dtype=torch.bool)
    mask[5:20] = False
    dirty = logits.clone()
    dirty[5:12], dirty[12:20] = NAN, INF
    ids[5:20] = 1 << 20
    w2, dw2 = w.clone(), dw.clone()
    w2[5:20] = dw2[5:20] = NAN
    counts, lse, losses = forward(eff, dirty, ids, mask)
    clean = check(eff, logits, ids, mask)
    assert all(torch.equal(a, b) for a, b in zip((counts, lse, losses), clean))
    out = torch.full((64, 32), NAN, device="cuda")
    eff.balance_loss_backward(dirty.cuda(), ids.cuda(), counts, lse, torch.tensor([1.0, 1.0], device="cuda"), out, w=w2.cuda(), dw=dw2.cuda())
    ref, err = B.balance_grad64(logits, torch.where(mask[:, None], ids, -1), counts.cpu().long(), lse.cpu(), torch.tensor([1.0, 1.0]), w, dw)
    R.assert_within(out, ref, err, "dlogits")
    assert not out[5:20].any()
    # experts that are masked, a row that is masked whole, and masks of the lowest value
    low = logits.clone()
    low[:, 7:20] = -INF
    low[3] = -INF
    low[9, 1:] = torch.finfo(F32).min
    low[10] = torch.finfo(F32).min
    ids = torch.topk(low, 4, dim=1)[1].to(I32)
    counts, lse, _ = check(eff, low, ids)
    assert int(counts[-1]) == 63
    check_grad(eff, low, ids, counts, lse, torch.tensor([1.0, 0.0]), w, dw)
    for dead in (torch.full((9, 32), -INF), torch.zeros(9, 32)):
        counts, lse, losses = forward(eff, dead, ids[:9], torch.zeros(9, dtype=torch.bool) if dead[0, 0] == 0 else None)
        assert not counts.any() and (lse == -INF).all() and not losses.any()
        out = torch.full((9, 32), NAN, device="cuda")
        eff.balance_loss_backward(dead.cuda(), ids[:9].cuda(), counts, lse, torch.ones(2, device="cuda"), out, w=w[:9].cuda(), dw=dw[:9].cuda())
        assert not out.any()


def test_no_tokens(eff):
    logits, ids = torch.empty(0, 12), torch.empty(0, 3, dtype=I32)
    counts, lse, losses = forward(eff, logits, ids)
    assert not counts.any() and not losses.any()
    eff.balance_loss_backward(logits.cuda(), ids.cuda(), counts, lse, torch.ones(2, device="cuda"), torch.empty(0, 12, device="cuda"))


def test_logits_that_are_no_numbers_show(eff):
    for bad in (NAN, INF):
        logits, ids, w, dw = batch(20, 16, 2, F32, 1)
        logits[4, 3] = bad
        counts, lse, losses = forward(eff, logits, ids)
        assert torch.isnan(losses).all() and int(counts[-1]) == 20
        logits[4] = bad
        assert torch.isnan(forward(eff, logits, ids)[2]).all()


def test_large_logits(eff):
    """The maximum is taken out first: nothing overflows at 1e4, in 16 bits either."""
    for dt in (F32, HF):
        logits, ids, w, dw = batch(30, 64, 4, dt, 2)
        logits = (logits.float() * 1000).to(dt)
        counts, lse, _ = check(eff, logits, ids)
        check_grad(eff, logits, ids, counts, lse, torch.tensor([1.0, 1e-6]), w, dw)


def test_strides(eff):
    """Rows apart and beginning at odd places; what lies between output rows stays."""
    full, ids, w, dw = batch(26, 90, 4, F32, 6)
    cu = full.cuda()
    for off, E in ((0, 64), (1, 64), (4, 80), (3, 77)):
        x = cu[::2, off:off + E]
        i = torch.where(ids[::2] < E, ids[::2], -1).contiguous()
        counts, lse, losses = check(eff, x.cpu(), i)
        again = forward(eff, x, i)
        for a, b, what in zip(again, (counts, lse, losses), ("counts", "lse", "losses")):
            torch.testing.assert_close(a, b, rtol=1e-5, atol=1e-5, msg=what)
        out = torch.full((13, 100), 5.0, device="cuda")
        eff.balance_loss_backward(x, i.cuda(), counts, lse, torch.ones(2, device="cuda"), out[:, off:off + E], w=w[::2].contiguous().cuda(), dw=dw[::2].contiguous().cuda())
        ref, err = B.balance_grad64(x.cpu(), i, counts.cpu().long(), lse.cpu(), torch.ones(2), w[::2], dw[::2])
        R.assert_within(out[:, off:off + E], ref, err, "dlogits")
        assert (out[:, :off] == 5).all() and (out[:, off + E:] == 5).all()


def test_an_even_load_is_one(eff):
    E, K = 32, 2
    logits = torch.zeros(64, E)
    ids = (torch.arange(128, dtype=I32) % E).view(64, K)
    _, _, losses = check(eff, logits, ids)
    assert abs(float(losses[0]) - 1) < 1e-6 and abs(float(losses[1]) - math.log(E) ** 2) < 1e-5


def test_the_gradients_are_the_formulas_derivatives():
    """The reference itself: against autograd of the losses' definition, and against differences."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(5, 6, generator=g, dtype=torch.float64, requires_grad=True)
    ids = torch.topk(x.detach(), 2, dim=1)[1]
    f = torch.bincount(ids.reshape(-1), minlength=6).double() / 10
    dw = torch.randn(5, 2, generator=g, dtype=torch.float64)

    def loss(x):
        lse = torch.logsumexp(x, 1)
        w = torch.softmax(x.gather(1, ids), 1)
        return 0.7 * 6 * (f * torch.softmax(x, 1).mean(0)).sum() - 0.2 * (lse ** 2).mean() + (w * dw).sum()

    assert torch.autograd.gradcheck(loss, (x,))
    want = torch.autograd.grad(loss(x), x)[0]
    with torch.no_grad():
        counts = torch.cat([f * 10, torch.tensor([5.0], dtype=torch.float64)]).long()
        got, _ = B.balance_grad64(x, ids, counts, torch.logsumexp(x, 1), torch.tensor([0.7, -0.2], dtype=torch.float64), torch.softmax(x.gather(1, ids), 1), dw)
    torch.testing.assert_close(got, want, rtol=1e-10, atol=1e-12)


def test_large_and_repeated(eff):
    """A long batch, the same bits from the same call, and losses against fp64."""
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn(100003, 128, generator=g, device="cuda")
    ids = torch.topk(logits, 4, dim=1)[1].to(I32)
    a, b = forward(eff, logits, ids), forward(eff, logits, ids)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    x = logits.double()
    f = torch.bincount(ids.reshape(-1).long(), minlength=128).double() / ids.numel()
    want = torch.stack([128 * (f * torch.softmax(x, 1).mean(0)).sum(), (torch.logsumexp(x, 1) ** 2).mean()])
    torch.testing.assert_close(a[2].double(), want, rtol=3e-6, atol=0)
