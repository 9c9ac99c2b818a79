"""What the operators without an engine refuse, before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    return e


A = 1 << 20    # stands for a device address: every call here is refused before it is used
OK = dict(dtype=0, out_dtype=0, act=0, groups=0, m=4, n=8, k=16, ld_x=16, ld_w=16, ld_y=8, ld_residual=8, ld_pre=8, stride_w=0,
          ld_dx=16, ld_dw=16, stride_dw=0)


def desc(**kw):
    from expert_ffn_serving_amd.ops import MatmulDesc
    return MatmulDesc(**{**OK, **kw})


def forward(eff, d, x=A, w=A, bias=None, residual=None, offsets=None, y=A, pre=None, ws=None, nws=0):
    return eff.lib().eff_matmul(None if d is None else ctypes.addressof(d), x, w, bias, residual, offsets, y, pre, ws, nws, None)


def backward(eff, d, dy=A, x=A, w=A, pre=None, offsets=None, dx=A, dw=A, dbias=A, ws=None, nws=0):
    return eff.lib().eff_matmul_backward(None if d is None else ctypes.addressof(d), dy, x, w, pre, offsets, dx, dw, dbias, ws, nws, None)


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(dtype=-1), dict(out_dtype=1), dict(out_dtype=7), dict(act=5), dict(act=-1),
                                dict(groups=-1), dict(groups=4097), dict(m=-1), dict(n=0), dict(k=0), dict(m=1 << 31),
                                dict(k=1 << 31), dict(n=1 << 31), dict(n=1 << 30, act=4)])
def test_bad_descriptions(eff, kw):
    d = desc(**kw)
    assert forward(eff, d) == eff.EFF_EINVAL
    assert backward(eff, d) == eff.EFF_EINVAL
    assert eff.lib().eff_matmul_workspace(ctypes.addressof(d), 0) == eff.EFF_EINVAL
    assert eff.lib().eff_last_error()


def test_bad_forward_calls(eff):
    assert forward(eff, None) == eff.EFF_EINVAL
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(offsets=A)):
        assert forward(eff, desc(), **kw) == eff.EFF_EINVAL, kw
    assert forward(eff, desc(groups=2)) == eff.EFF_EINVAL            # no offsets
    for kw in (dict(ld_x=-1), dict(ld_w=-16), dict(ld_residual=-1), dict(stride_w=-1), dict(ld_y=7)):
        assert forward(eff, desc(**kw)) == eff.EFF_EINVAL, kw
    assert forward(eff, desc(ld_pre=7), pre=A) == eff.EFF_EINVAL
    big = desc(m=1 << 30, n=1 << 20, ld_y=1 << 20, ld_residual=1 << 20, ld_pre=1 << 20)
    assert forward(eff, big) == eff.EFF_EINVAL                        # more tiles than a grid holds
    big = desc(m=1 << 30, n=1 << 12, k=1 << 12, ld_x=1 << 12, ld_w=1 << 12, ld_y=1 << 12, ld_dx=1 << 12, ld_dw=1 << 12)
    ws = eff.lib().eff_matmul_workspace(ctypes.addressof(big), 1)
    assert backward(eff, big, ws=A, nws=ws) == eff.EFF_EINVAL
    assert forward(eff, desc(m=0), x=None, y=None) == eff.EFF_OK      # no rows: nothing to do


def test_bad_backward_calls(eff):
    assert backward(eff, None) == eff.EFF_EINVAL
    for kw in (dict(dy=None), dict(x=None), dict(w=None), dict(offsets=A)):
        assert backward(eff, desc(), **kw) == eff.EFF_EINVAL, kw
    assert backward(eff, desc(act=1)) == eff.EFF_EINVAL               # no pre
    assert backward(eff, desc(act=1), pre=A) == eff.EFF_EINVAL        # no workspace
    d = desc(act=1)
    need = eff.lib().eff_matmul_workspace(ctypes.addressof(d), 1)
    assert need > 0 and need % 256 == 0
    assert backward(eff, desc(act=1), pre=A, ws=A, nws=need - 1) == eff.EFF_EINVAL
    assert backward(eff, desc(act=1), pre=A, ws=A + 16, nws=need) == eff.EFF_EINVAL
    for kw in (dict(ld_dx=15), dict(ld_dw=15), dict(ld_y=-1), dict(groups=2, stride_w=128, stride_dw=127)):
        assert backward(eff, desc(**kw), offsets=A if kw.get("groups") else None) == eff.EFF_EINVAL, kw


def test_bad_token_calls(eff):
    L = eff.lib()
    assert L.eff_sort_tokens_workspace(-1, 4) == eff.EFF_EINVAL
    assert L.eff_sort_tokens_workspace(1 << 31, 4) == eff.EFF_EINVAL
    for E in (0, -1, 4097):
        assert L.eff_sort_tokens_workspace(10, E) == eff.EFF_EINVAL
        assert L.eff_sort_tokens(A, 10, E, A, A, A, None, 0, None) == eff.EFF_EINVAL
    for args in ((None, 10, 4, A, A, A), (A, 10, 4, None, A, A), (A, 10, 4, A, None, A), (A, 10, 4, A, A, None)):
        assert L.eff_sort_tokens(*args, None, 0, None) == eff.EFF_EINVAL
    need = L.eff_sort_tokens_workspace(1 << 20, 256)
    assert need > 0
    assert L.eff_sort_tokens(A, 1 << 20, 256, A, A, A, A, need - 1, None) == eff.EFF_EINVAL
    good = dict(dtype=0, T=4, K=2, H=8, rows=8)
    for kw in (dict(dtype=3), dict(dtype=-1), dict(T=-1), dict(K=0), dict(K=33), dict(H=0), dict(rows=-1), dict(T=1 << 30, K=2),
               dict(H=1 << 31), dict(rows=1 << 31)):
        a = {**good, **kw}
        dt, T, K, H, rows = (a[i] for i in ("dtype", "T", "K", "H", "rows"))
        assert L.eff_dispatch_tokens(dt, A, 8, A, T, K, H, A, 8, rows, None) == eff.EFF_EINVAL, kw
        assert L.eff_dispatch_tokens_backward(dt, A, 8, rows, A, T, K, H, A, 8, None) == eff.EFF_EINVAL, kw
        assert L.eff_combine_tokens(dt, A, 8, rows, A, A, T, K, H, None, 0, A, 8, None) == eff.EFF_EINVAL, kw
        assert L.eff_combine_tokens_backward(dt, A, 8, A, 8, rows, A, A, T, K, H, A, 8, A, None) == eff.EFF_EINVAL, kw
    for x, p, xs, ldx, lds in ((None, A, A, 8, 8), (A, None, A, 8, 8), (A, A, None, 8, 8), (A, A, A, -8, 8), (A, A, A, 8, 7)):
        assert L.eff_dispatch_tokens(0, x, ldx, p, 4, 2, 8, xs, lds, 8, None) == eff.EFF_EINVAL
        assert L.eff_dispatch_tokens_backward(0, x, ldx, 8, p, 4, 2, 8, xs, lds, None) == eff.EFF_EINVAL
        assert L.eff_combine_tokens(0, x, ldx, 8, p, A, 4, 2, 8, None, 0, xs, lds, None) == eff.EFF_EINVAL
        assert L.eff_combine_tokens_backward(0, A, 8, x, ldx, 8, p, A, 4, 2, 8, xs, lds, A, None) == eff.EFF_EINVAL
    assert L.eff_combine_tokens(0, A, 8, 8, A, None, 4, 2, 8, None, 0, A, 8, None) == eff.EFF_EINVAL
    assert L.eff_combine_tokens(0, A, 8, 8, A, A, 4, 2, 8, A, -1, A, 8, None) == eff.EFF_EINVAL


def test_tensors_that_are_not_on_the_gpu(eff):
    x, w, y = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(6, 8, dtype=torch.bfloat16), torch.zeros(4, 6, dtype=torch.bfloat16)
    i32 = torch.zeros(4, 2, dtype=torch.int32)
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: eff.matmul(x, w, y), lambda: eff.matmul_backward(y, x, w, dx=x), lambda: eff.grouped_matmul(x, w[None], off, y),
                 lambda: eff.grouped_matmul(x, w[None], None, y), lambda: eff.grouped_matmul_backward(y, x, w[None], None),
                 lambda: eff.sort_tokens(i32, off, i32.view(-1), i32), lambda: eff.dispatch_tokens(x, i32, y),
                 lambda: eff.dispatch_tokens_backward(x, i32, y), lambda: eff.combine_tokens(x, i32, None, y),
                 lambda: eff.combine_tokens_backward(x, x, i32, None, x), lambda: eff.matmul(None, w, y)):
        with pytest.raises(eff.EffError) as ei:
            call()
        assert ei.value.code == eff.EFF_EINVAL


@pytest.mark.gpu
def test_bad_tensors(eff):
    z = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    x, w, y = z(4, 16), z(8, 16), z(4, 8)
    pos, ids, off = z(4, 2, d=torch.int32), z(4, 2, d=torch.int32), z(3, d=torch.int32)
    fw, hf = z(4, 2, d=torch.float32), torch.float16
    calls = [
        lambda: eff.matmul(x.float(), w, y), lambda: eff.matmul(x, w.half(), y), lambda: eff.matmul(x, w, y.half()),
        lambda: eff.matmul(x[0], w, y), lambda: eff.matmul(x, w, z(4, 9)), lambda: eff.matmul(x, z(8, 15), y),
        lambda: eff.matmul(x, w, y, bias=z(7)), lambda: eff.matmul(x, w, y, bias=z(16)[::2]),
        lambda: eff.matmul(x, w, y, residual=z(4, 7)), lambda: eff.matmul(x, w, y, residual=z(4, 8, d=hf)),
        lambda: eff.matmul(x, w, y, pre=z(4, 7)), lambda: eff.matmul(x, w, y, act=9),
        lambda: eff.matmul(x, z(7, 16), z(4, 3), act=eff.ACT_SWIGLU), lambda: eff.matmul(z(16, 4).t(), w, y),
        lambda: eff.matmul(x, w, z(1, 8).expand(4, 8)), lambda: eff.matmul(x, w, y.cpu()), lambda: eff.matmul(x, w.cpu(), y),
        lambda: eff.matmul_backward(y, x, w, dx=z(4, 15)), lambda: eff.matmul_backward(y, x, w, dw=z(8, 15)),
        lambda: eff.matmul_backward(y, x, w, dbias=z(9)), lambda: eff.matmul_backward(y, x, w, dx=x, act=eff.ACT_SILU),
        lambda: eff.matmul_backward(y.half(), x, w, dx=x), lambda: eff.matmul_backward(y, x, w, dx=z(1, 16).expand(4, 16)),
        lambda: eff.grouped_matmul(x, w, off, y), lambda: eff.grouped_matmul(x, z(2, 8, 16), z(2, d=torch.int32), y),
        lambda: eff.grouped_matmul(x, z(2, 8, 16), off.long(), y), lambda: eff.grouped_matmul(x, z(2, 8, 16), off.cpu(), y),
        lambda: eff.grouped_matmul_backward(y, x, z(2, 8, 16), off, dw=z(1, 8, 16).expand(2, 8, 16)),
        lambda: eff.grouped_matmul(x, z(0, 8, 16), z(1, d=torch.int32), y), lambda: eff.grouped_matmul(x, z(2, 8, 32)[..., ::2], off, y),
        lambda: eff.matmul(x, None, y), lambda: eff.matmul(x, w, None), lambda: eff.matmul(x, w, y, bias=3), lambda: eff.matmul(x, w, y, residual="r"),
        lambda: eff.matmul(x, w, y, pre=y.cpu().float().numpy()), lambda: eff.matmul_backward(None, x, w), lambda: eff.dispatch_tokens(x, None, x),
        lambda: eff.sort_tokens(ids, None, ids.view(-1), pos), lambda: eff.combine_tokens(z(8, 16), pos, None, x),
        lambda: eff.sort_tokens(ids.long(), off, ids.view(-1), pos), lambda: eff.sort_tokens(ids, off, z(7, d=torch.int32), pos),
        lambda: eff.sort_tokens(ids, off, ids.view(-1), z(2, 4, d=torch.int32)), lambda: eff.sort_tokens(ids, off[:1], ids.view(-1), pos),
        lambda: eff.sort_tokens(ids, z(4098, d=torch.int32), z(8, d=torch.int32), pos), lambda: eff.sort_tokens(ids.t(), off, z(8, d=torch.int32), pos),
        lambda: eff.dispatch_tokens(x, pos, z(8, 15)), lambda: eff.dispatch_tokens(x, pos, z(8, 16, d=hf)),
        lambda: eff.dispatch_tokens(x, pos[:3], z(8, 16)), lambda: eff.dispatch_tokens(x, z(4, 33, d=torch.int32), z(8, 16)),
        lambda: eff.dispatch_tokens(x.int(), pos, z(8, 16)), lambda: eff.dispatch_tokens(x, pos.long(), z(8, 16)),
        lambda: eff.dispatch_tokens_backward(z(8, 16), pos, z(4, 15)), lambda: eff.dispatch_tokens_backward(z(8, 16), pos, z(3, 16)),
        lambda: eff.combine_tokens(z(8, 16), pos, fw.half(), x), lambda: eff.combine_tokens(z(8, 16), pos, z(4, 3, d=torch.float32), x),
        lambda: eff.combine_tokens(z(8, 16), pos, fw, x, residual=z(4, 15)), lambda: eff.combine_tokens(z(8, 16), pos, fw.cpu(), x),
        lambda: eff.combine_tokens_backward(x, z(8, 16), pos, fw, z(7, 16)), lambda: eff.combine_tokens_backward(x, z(8, 16), pos, fw, z(8, 16), z(4, 2)),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(eff.EffError) as ei:
            call()
        assert ei.value.code == eff.EFF_EINVAL, i
