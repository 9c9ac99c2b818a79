"""The operators beside torch's autograd: they record nothing, and what they write counts as written in place, so that a graph
that saved such a tensor refuses its backward pass instead of using the new values."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    return e


def calls(eff):
    """name -> (call, outputs)."""
    z = lambda *s, d=BF: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    x, w, w3, off = z(4, 16), z(8, 16), z(2, 8, 16), torch.tensor([0, 1, 4], dtype=I32, device="cuda")
    y, pre, dx, dw, db, dw3, db2 = z(4, 8), z(4, 8), z(4, 16), z(8, 16), z(8), z(2, 8, 16), z(2, 8)
    ids, pos, order, o3 = z(4, 2, d=I32), z(4, 2, d=I32), z(8, d=I32), z(3, d=I32)
    places = torch.arange(8, dtype=I32, device="cuda").view(4, 2)
    rows, out, gate, dgate = z(8, 16), z(4, 16), z(4, 2, d=F32), z(4, 2, d=F32)
    return {
        "matmul": (lambda: eff.matmul(x, w, y, act=eff.ACT_SILU, pre=pre), [y, pre]),
        "grouped_matmul": (lambda: eff.grouped_matmul(x, w3, off, y, pre=pre), [y, pre]),
        "matmul_backward": (lambda: eff.matmul_backward(y, x, w, dx=dx, dw=dw, dbias=db), [dx, dw, db]),
        "grouped_matmul_backward": (lambda: eff.grouped_matmul_backward(y, x, w3, off, dx=dx, dw=dw3, dbias=db2), [dx, dw3, db2]),
        "sort_tokens": (lambda: eff.sort_tokens(ids, o3, order, pos), [o3, order, pos]),
        "dispatch_tokens": (lambda: eff.dispatch_tokens(x, places, rows), [rows]),
        "dispatch_tokens_backward": (lambda: eff.dispatch_tokens_backward(rows, places, dx), [dx]),
        "combine_tokens": (lambda: eff.combine_tokens(rows, places, gate, out, residual=x), [out]),
        "combine_tokens_backward": (lambda: eff.combine_tokens_backward(out, x.repeat(2, 1), places, gate, rows, dgate), [rows, dgate]),
    }


NAMES = ["matmul", "grouped_matmul", "matmul_backward", "grouped_matmul_backward", "sort_tokens", "dispatch_tokens",
         "dispatch_tokens_backward", "combine_tokens", "combine_tokens_backward"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_count_as_written(eff, name):
    call, outs = calls(eff)[name]
    before = [t._version for t in outs]
    call()
    assert all(t._version > v for t, v in zip(outs, before))


def test_a_graph_that_saved_an_output_refuses_its_backward(eff):
    a = torch.ones(4, 8, dtype=BF, device="cuda", requires_grad=True)
    x, w, y = torch.ones(4, 16, dtype=BF, device="cuda"), torch.ones(8, 16, dtype=BF, device="cuda"), torch.ones(4, 8, dtype=BF, device="cuda")
    kept = (a * y).sum()
    eff.matmul(x, w, y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        kept.backward()
    (a * y).sum().backward()
    assert (a.grad == 16).all()


def test_inputs_that_require_grad_and_inference_tensors(eff):
    x = torch.ones(4, 16, dtype=BF, device="cuda", requires_grad=True)
    w, y = torch.nn.Parameter(torch.ones(8, 16, dtype=BF, device="cuda")), torch.empty(4, 8, dtype=BF, device="cuda")
    eff.matmul(x, w, y)
    assert not y.requires_grad and y.grad_fn is None and (y == 16).all()
    with torch.inference_mode():
        x, w, y = torch.ones(4, 16, dtype=BF, device="cuda"), torch.ones(8, 16, dtype=BF, device="cuda"), torch.empty(4, 8, dtype=BF, device="cuda")
        eff.matmul(x, w, y)
    eff.matmul(x, w, y)
    assert (y == 16).all()
