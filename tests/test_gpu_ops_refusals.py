"""Arguments that the binding refuses before it calls the library: counts that do not fit the library's 32-bit ones, values of
the wrong kind, a stream of another device."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    yield e
    torch.cuda.empty_cache()


def refused(eff, call):
    with pytest.raises(eff.EffError) as ei:
        call()
    assert ei.value.code == eff.EFF_EINVAL


def test_counts_beyond_32_bits(eff):
    """2^32 + 1 places a token or experts are not 1."""
    many = (1 << 32) + 1
    x, xs = torch.ones(1, 8, dtype=BF, device="cuda"), torch.zeros(4, 8, dtype=BF, device="cuda")
    pos = torch.empty(1, many, dtype=I32, device="cuda")
    pos[0, 0] = 1
    refused(eff, lambda: eff.dispatch_tokens(x, pos, xs))
    refused(eff, lambda: eff.dispatch_tokens_backward(xs, pos, x))
    assert (x == 1).all() and not xs.any()
    offsets, ids, order, place = pos.view(-1), torch.zeros(4, dtype=I32, device="cuda"), torch.zeros(4, dtype=I32, device="cuda"), \
        torch.zeros(4, dtype=I32, device="cuda")
    refused(eff, lambda: eff.sort_tokens(ids, torch.empty(many + 1, dtype=I32, device="cuda"), order, place))
    w, y = torch.ones(1, 8, 8, dtype=BF, device="cuda").expand(1 << 32, 8, 8), torch.zeros(1, 8, dtype=BF, device="cuda")
    refused(eff, lambda: eff.grouped_matmul(x, w, offsets, y))
    assert not y.any()


def test_values_of_another_kind(eff):
    x, w, y = (torch.ones(s, dtype=BF, device="cuda") for s in ((4, 16), (8, 16), (4, 8)))
    for act in (1.0, 4.0, "silu", None):
        refused(eff, lambda: eff.matmul(x, w, y, act=act))
        refused(eff, lambda: eff.matmul_backward(y, x, w, dx=torch.empty_like(x), act=act, pre=y))
    for stream in ("s", 1.5):
        refused(eff, lambda: eff.matmul(x, w, y, stream=stream))


def test_stream_of_another_device(eff):
    class Stream:
        cuda_stream, device_index = torch.cuda.current_stream().cuda_stream, 1

    x, w, y = (torch.ones(s, dtype=BF, device="cuda") for s in ((4, 16), (8, 16), (4, 8)))
    refused(eff, lambda: eff.matmul(x, w, y, stream=Stream()))
    eff.matmul(x, w, y, stream=torch.cuda.current_stream())
    assert (y == 16).all()
