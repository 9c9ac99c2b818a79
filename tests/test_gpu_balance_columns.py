"""The router's losses where the partial sums of the columns are many (parts x (E + 1) above 65536): several workgroups add them up
before the one that computes the losses.  That the sizes lie where they should is worked out beside them."""
import pytest
import torch

from tests.test_gpu_balance import batch, check, check_grad

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    return e


def sums(T, E):
    """Partial sums: a row of E + 1 for every workgroup, each with 16 waves (4 beyond 1024 experts) of two rows and more, at most 256."""
    W = 16 if E <= 1024 else 4
    return (1 if T <= 4 * W else min(256, -(-T // (2 * W)))) * (E + 1)


# E below and beyond 1024, few parts and all 256, E + 1 a multiple of 64 and not, either side of 65536
@pytest.mark.parametrize("T,E,dt,above", [(9000, 257, F32, True), (8200, 319, BF, True), (2600, 1000, HF, True), (512, 4096, F32, True),
                                          (300, 2050, BF, True), (130, 4095, F32, True), (2100, 1100, F32, True),
                                          (8192, 255, F32, False), (8193, 256, F32, True), (127, 4095, BF, False), (129, 4095, BF, True)])
def test_many_partial_sums(eff, T, E, dt, above):
    assert (sums(T, E) > 65536) == above
    logits, ids, w, dw = batch(T, E, 4, dt, T + E)
    mask = torch.rand(T, generator=torch.Generator().manual_seed(E)) > 0.3
    counts, lse, losses = check(eff, logits, ids, mask)
    again = check(eff, logits, ids, mask)
    assert all(torch.equal(a, b) for a, b in zip((counts, lse, losses), again))
    if T <= 600:
        check_grad(eff, logits, ids, counts, lse, torch.tensor([1e-2, 1e-3]), w, dw)


def test_all_but_one_masked(eff):
    """One live token among many parts, and none."""
    logits, ids, _, _ = batch(9000, 300, 3, F32, 1)
    mask = torch.zeros(9000, dtype=torch.bool)
    counts, _, losses = check(eff, logits, ids, mask)
    assert not counts.any() and not losses.any()
    mask[8999] = True
    counts, _, _ = check(eff, logits, ids, mask)
    assert int(counts[-1]) == 1


def test_logits_that_are_no_numbers_show(eff):
    for bad in (float("nan"), float("inf")):
        logits, ids, _, _ = batch(512, 4096, 2, F32, 2)
        logits[511, 4095] = bad
        counts = torch.empty(4097, dtype=torch.int32, device="cuda")
        lse, losses = torch.empty(512, device="cuda"), torch.empty(2, device="cuda")
        eff.balance_loss(logits.cuda(), ids.cuda(), counts, lse, losses)
        assert torch.isnan(losses).all() and int(counts[-1]) == 512
        assert torch.isfinite(lse[:511]).all() and not torch.isfinite(lse[511])
