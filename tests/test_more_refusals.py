"""What layer norm, the router's losses, 4-bit rows and their products refuse, before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    return e


A = 1 << 20    # stands for a device address: every call here is refused before it is used
NAN, INF = float("nan"), float("inf")


def test_layer_norm(eff):
    L = eff.lib()
    good = dict(dt=0, wt=0, x=A, ldx=8, w=A, b=A, eps=1e-5, T=4, H=8, y=A, ldy=8, mean=A, rstd=A)

    def call(**kw):
        a = {**good, **kw}
        return L.eff_layer_norm(a["dt"], a["wt"], a["x"], a["ldx"], a["w"], a["b"], a["eps"], a["T"], a["H"], a["y"], a["ldy"], a["mean"], a["rstd"], None)

    for kw in (dict(dt=3), dict(dt=-1), dict(wt=1), dict(dt=2, wt=0), dict(wt=3), dict(T=-1), dict(T=1 << 31), dict(H=0), dict(H=1 << 31),
               dict(x=None), dict(y=None), dict(ldx=-1), dict(ldy=7), dict(eps=-1e-5), dict(eps=NAN), dict(eps=INF)):
        assert call(**kw) == eff.EFF_EINVAL, kw
    assert call(T=0, x=None, y=None) == eff.EFF_OK
    ok = dict(dt=0, wt=0, dy=A, lddy=8, x=A, ldx=8, w=A, mean=A, rstd=A, res=None, ldr=0, T=4, H=8, dx=A, lddx=8, dw=A, db=A, ws=A, n=1 << 20)

    def back(**kw):
        a = {**ok, **kw}
        return L.eff_layer_norm_backward(*[a[i] for i in ("dt", "wt", "dy", "lddy", "x", "ldx", "w", "mean", "rstd", "res", "ldr", "T", "H", "dx",
                                                          "lddx", "dw", "db", "ws", "n")], None)

    need = L.eff_layer_norm_backward_workspace(4, 8)
    assert need > 0 and need % 256 == 0
    for kw in (dict(dt=3), dict(wt=1), dict(T=-1), dict(H=0), dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(lddy=-1),
               dict(ldx=-1), dict(ldr=-1), dict(lddx=7), dict(ws=None), dict(n=need - 1), dict(ws=A + 16)):
        assert back(**kw) == eff.EFF_EINVAL, kw
    assert back(dx=None, dw=None, db=None, ws=None, n=0) == eff.EFF_OK
    assert back(T=0, dw=None, db=None, ws=None, n=0) == eff.EFF_OK
    assert L.eff_layer_norm_backward_workspace(-1, 8) == eff.EFF_EINVAL and L.eff_layer_norm_backward_workspace(4, 0) == eff.EFF_EINVAL


def test_balance(eff):
    L = eff.lib()
    need = L.eff_balance_loss_workspace(4, 16)
    assert need > 0 and need % 256 == 0
    for T, E in ((-1, 4), (1 << 31, 4), (4, 0), (4, 4097)):
        assert L.eff_balance_loss_workspace(T, E) == eff.EFF_EINVAL
    good = dict(dt=2, x=A, ld=16, ids=A, mask=None, T=4, K=2, E=16, counts=A, lse=A, losses=A, ws=A, n=need)

    def call(**kw):
        a = {**good, **kw}
        return L.eff_balance_loss(*[a[i] for i in ("dt", "x", "ld", "ids", "mask", "T", "K", "E", "counts", "lse", "losses", "ws", "n")], None)

    for kw in (dict(dt=3), dict(dt=-1), dict(T=-1), dict(K=0), dict(K=33), dict(E=0), dict(E=4097), dict(T=1 << 30), dict(x=None), dict(ids=None),
               dict(counts=None), dict(lse=None), dict(losses=None), dict(ld=-1), dict(ws=None), dict(n=need - 1), dict(ws=A + 8)):
        assert call(**kw) == eff.EFF_EINVAL, kw
    ok = dict(dt=2, x=A, ld=16, ids=A, counts=A, lse=A, dl=A, w=A, dw=A, T=4, K=2, E=16, out=A, ldd=16)

    def back(**kw):
        a = {**ok, **kw}
        return L.eff_balance_loss_backward(*[a[i] for i in ("dt", "x", "ld", "ids", "counts", "lse", "dl", "w", "dw", "T", "K", "E", "out", "ldd")], None)

    for kw in (dict(dt=3), dict(T=-1), dict(K=0), dict(K=33), dict(E=0), dict(E=4097), dict(x=None), dict(ids=None), dict(counts=None),
               dict(lse=None), dict(out=None), dict(w=None), dict(dw=None), dict(ld=-1), dict(ldd=15)):
        assert back(**kw) == eff.EFF_EINVAL, kw
    assert back(T=0, x=None) == eff.EFF_OK


def test_rows(eff):
    L = eff.lib()
    assert L.eff_mx4_code_bytes(1) == 64 and L.eff_mx4_scale_bytes(1) == 4 and L.eff_mx4_code_bytes(2560) == 1280 and L.eff_mx4_scale_bytes(129) == 8
    assert eff.mx4_row_bytes(2563) == (L.eff_mx4_code_bytes(2563), L.eff_mx4_scale_bytes(2563))
    for k in (0, -1, 1 << 31):
        assert L.eff_mx4_code_bytes(k) == eff.EFF_EINVAL and L.eff_mx4_scale_bytes(k) == eff.EFF_EINVAL
    good = dict(dt=0, x=A, ldx=200, rows=4, k=200, c=A, ldc=128, s=A, lds=8)

    def both(want, **kw):
        a = {**good, **kw}
        assert L.eff_mx4_quantize(*[a[i] for i in ("dt", "x", "ldx", "rows", "k", "c", "ldc", "s", "lds")], None) == want, kw
        assert L.eff_mx4_dequantize(*[a[i] for i in ("dt", "c", "ldc", "s", "lds", "rows", "k", "x", "ldx")], None) == want, kw

    for kw in (dict(dt=3), dict(dt=-1), dict(rows=-1), dict(rows=1 << 31), dict(k=0), dict(k=1 << 31), dict(x=None), dict(c=None), dict(s=None),
               dict(c=A + 8), dict(s=A + 2), dict(ldc=136), dict(lds=10), dict(ldx=-1)):
        both(eff.EFF_EINVAL, **kw)
    both(eff.EFF_OK, rows=0, x=None)
    assert L.eff_mx4_quantize(0, A, 200, 4, 200, A, 112, A, 8, None) == eff.EFF_EINVAL      # rows of an output overlap
    assert L.eff_mx4_quantize(0, A, 200, 4, 200, A, 128, A, 4, None) == eff.EFF_EINVAL
    assert L.eff_mx4_dequantize(0, A, 128, A, 8, 4, 200, A, 199, None) == eff.EFF_EINVAL


OK = dict(x_dtype=3, dtype=0, out_dtype=0, act=0, groups=0, m=4, n=8, k=256, ld_x=128, ld_xs=8, ld_w=128, ld_ws=8, stride_w=1024, stride_ws=64,
          ld_y=8, ld_residual=8, ld_pre=8)


def product(eff, d, x=A, xs=A, w=A, ws=A, bias=None, residual=None, offsets=None, y=A, pre=None, tmp=None, n=0):
    return eff.lib().eff_mx4_matmul(None if d is None else ctypes.addressof(d), x, xs, w, ws, bias, residual, offsets, y, pre, tmp, n, None)


def desc(**kw):
    from expert_ffn_serving_amd.ops import Mx4Desc
    return Mx4Desc(**{**OK, **kw})


def test_products(eff):
    L = eff.lib()
    for kw in (dict(dtype=2), dict(dtype=3), dict(x_dtype=1), dict(x_dtype=2), dict(x_dtype=4), dict(out_dtype=1), dict(act=5), dict(act=-1),
               dict(groups=-1), dict(groups=4097), dict(reserved=1), dict(m=-1), dict(m=1 << 31), dict(n=0), dict(n=1 << 31), dict(k=0),
               dict(k=1 << 31), dict(n=1 << 30, act=4)):
        assert product(eff, desc(**kw)) == eff.EFF_EINVAL, kw
        assert L.eff_mx4_matmul_workspace(ctypes.addressof(desc(**kw))) == eff.EFF_EINVAL, kw
    assert product(eff, None) == eff.EFF_EINVAL
    for kw in (dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(y=None), dict(offsets=A), dict(x=A + 8), dict(w=A + 8), dict(xs=A + 2),
               dict(ws=A + 1)):
        assert product(eff, desc(), **kw) == eff.EFF_EINVAL, kw
    for kw in (dict(ld_x=-128), dict(ld_w=-128), dict(ld_xs=-8), dict(ld_ws=-8), dict(ld_x=136), dict(ld_w=136), dict(ld_xs=9), dict(ld_ws=10),
               dict(ld_residual=-1), dict(ld_y=7)):
        assert product(eff, desc(**kw)) == eff.EFF_EINVAL, kw
    assert product(eff, desc(groups=2)) == eff.EFF_EINVAL                 # no offsets
    for kw in (dict(stride_w=1032), dict(stride_ws=66), dict(stride_w=-1024)):
        assert product(eff, desc(groups=2, **kw), offsets=A) == eff.EFF_EINVAL, kw
    assert product(eff, desc(ld_pre=7), pre=A) == eff.EFF_EINVAL
    assert product(eff, desc(out_dtype=2), residual=A) == eff.EFF_EINVAL  # in place, of another type
    assert product(eff, desc(ld_residual=16), residual=A) == eff.EFF_EINVAL
    assert L.eff_mx4_matmul_workspace(ctypes.addressof(desc())) == 0 and L.eff_mx4_matmul_workspace(ctypes.addressof(desc(x_dtype=0, ld_x=256))) == 0
    assert product(eff, desc(x_dtype=0, ld_x=256)) == eff.EFF_EINVAL      # xs with 16-bit x
    d = desc(m=4000, x_dtype=0, ld_x=256, ld_xs=0)                         # more rows than the kernel quantises itself
    need = L.eff_mx4_matmul_workspace(ctypes.addressof(d))
    assert need >= 4000 * 128 + 4000 * 8 and need % 256 == 0
    assert product(eff, d) == eff.EFF_EINVAL                               # xs with 16-bit x
    for kw in (dict(tmp=None, n=need), dict(tmp=A, n=need - 1), dict(tmp=A + 16, n=need)):
        assert product(eff, d, xs=None, **kw) == eff.EFF_EINVAL, kw
    assert product(eff, desc(m=(1 << 31) - 1, n=1 << 29, ld_y=1 << 29)) == eff.EFF_EINVAL     # more tiles than a grid holds
    assert product(eff, desc(m=0), x=None, xs=None, y=None) == eff.EFF_OK


def test_tensors_that_are_not_on_the_gpu(eff):
    x, f, i32, u8 = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 64, dtype=torch.uint8)
    for call in (lambda: eff.layer_norm(x, x), lambda: eff.layer_norm_backward(x, x, f, f), lambda: eff.balance_loss(x, i32, i32, f, f),
                 lambda: eff.balance_loss_backward(x, i32, i32, f, f, x), lambda: eff.mx4_quantize(x, u8, u8), lambda: eff.mx4_dequantize(u8, u8, x),
                 lambda: eff.mx4_matmul(x, u8, u8, x), lambda: eff.grouped_mx4_matmul(x, u8, u8, i32, x), lambda: eff.grouped_mx4_matmul(x, u8, u8, None, x),
                 lambda: eff.layer_norm(None, x), lambda: eff.mx4_quantize(None, u8, u8), lambda: eff.mx4_matmul("x", u8, u8, x)):
        with pytest.raises(eff.EffError) as ei:
            call()
        assert ei.value.code == eff.EFF_EINVAL


@pytest.mark.gpu
def test_bad_tensors(eff):
    z = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    F32, HF, I32, U8 = torch.float32, torch.float16, torch.int32, torch.uint8
    x, y, w, s4 = z(4, 256), z(4, 256), z(256), z(4, d=F32)
    lg, ids, cn, ls = z(4, 16, d=F32), z(4, 2, d=I32), z(17, d=I32), z(2, d=F32)
    gw = z(4, 2, d=F32)
    c, sc, wq, ws, out = z(4, 128, d=U8), z(4, 8, d=U8), z(6, 128, d=U8), z(6, 8, d=U8), z(4, 6)
    w3, ws3, off = z(2, 6, 128, d=U8), z(2, 6, 8, d=U8), z(3, d=I32)
    calls = [
        lambda: eff.layer_norm(x, z(4, 255)), lambda: eff.layer_norm(x, y.half()), lambda: eff.layer_norm(x.int(), y), lambda: eff.layer_norm(x[0], y[0]),
        lambda: eff.layer_norm(x, y, weight=z(255)), lambda: eff.layer_norm(x, y, weight=z(256, d=HF)), lambda: eff.layer_norm(x, y, weight=w, bias=z(256, d=F32)),
        lambda: eff.layer_norm(x, y, weight=z(512)[::2]), lambda: eff.layer_norm(x, y, mean=z(4)), lambda: eff.layer_norm(x, y, rstd=z(3, d=F32)),
        lambda: eff.layer_norm(x, y, eps=-1.0), lambda: eff.layer_norm(x, y, eps="a"), lambda: eff.layer_norm(x, y, eps=None), lambda: eff.layer_norm(x, y, eps=NAN),
        lambda: eff.layer_norm(x, z(1, 256).expand(4, 256)), lambda: eff.layer_norm(x, y.cpu()), lambda: eff.layer_norm(x, None), lambda: eff.layer_norm(x, y, weight=1.0),
        lambda: eff.layer_norm(z(256, 4).t(), y), lambda: eff.layer_norm_backward(x, x, s4, s4, dx=z(4, 255)), lambda: eff.layer_norm_backward(x, x, s4, s4, dw=z(255)),
        lambda: eff.layer_norm_backward(x, x, s4, s4, dw=z(256, d=HF)), lambda: eff.layer_norm_backward(x, x, s4, s4, dw=w, db=z(256, d=F32)),
        lambda: eff.layer_norm_backward(x, x, s4, s4, dw=z(256, d=F32), weight=w), lambda: eff.layer_norm_backward(x.half(), x, s4, s4, dx=y),
        lambda: eff.layer_norm_backward(x, x, s4.half(), s4, dx=y), lambda: eff.layer_norm_backward(x, x, None, s4, dx=y),
        lambda: eff.layer_norm_backward(x, x, s4, s4, dx=y, residual=z(4, 255)), lambda: eff.layer_norm_backward(x, x, s4, s4, dx=y, residual=y.half()),
        lambda: eff.balance_loss(lg, ids, cn[:16], s4, ls), lambda: eff.balance_loss(lg, ids.long(), cn, s4, ls), lambda: eff.balance_loss(lg, ids[:3], cn, s4, ls),
        lambda: eff.balance_loss(lg, ids, cn, s4.half(), ls), lambda: eff.balance_loss(lg, ids, cn, s4, z(3, d=F32)), lambda: eff.balance_loss(lg.double(), ids, cn, s4, ls),
        lambda: eff.balance_loss(lg, ids, cn, s4, ls, mask=z(4, d=U8)), lambda: eff.balance_loss(lg, ids, cn, s4, ls, mask=z(3, d=torch.bool)),
        lambda: eff.balance_loss(lg, z(4, 33, d=I32), cn, s4, ls), lambda: eff.balance_loss(z(4, 4097, d=F32), ids, z(4098, d=I32), s4, ls),
        lambda: eff.balance_loss(z(4, 0, d=F32), ids, z(1, d=I32), s4, ls), lambda: eff.balance_loss(lg, ids, cn, None, ls),
        lambda: eff.balance_loss_backward(lg, ids, cn, s4, ls, lg.half()), lambda: eff.balance_loss_backward(lg, ids, cn, s4, ls, z(4, 15, d=F32)),
        lambda: eff.balance_loss_backward(lg, ids, cn, s4, ls, lg.clone(), w=gw), lambda: eff.balance_loss_backward(lg, ids, cn, s4, ls, lg.clone(), dw=gw),
        lambda: eff.balance_loss_backward(lg, ids, cn, s4, ls, lg.clone(), w=gw, dw=gw.half()), lambda: eff.balance_loss_backward(lg, ids, cn, s4, s4, lg.clone()),
        lambda: eff.balance_loss_backward(lg, ids, cn, s4, ls, z(1, 16, d=F32).expand(4, 16)), lambda: eff.balance_loss_backward(lg, ids, None, s4, ls, lg.clone()),
        lambda: eff.mx4_quantize(x, c[:3], sc), lambda: eff.mx4_quantize(x, z(4, 64, d=U8), sc), lambda: eff.mx4_quantize(x, c, z(4, 4, d=U8)),
        lambda: eff.mx4_quantize(x, c.char(), sc), lambda: eff.mx4_quantize(x.int(), c, sc), lambda: eff.mx4_quantize(x, z(4, 136, d=U8)[:, :128], sc),
        lambda: eff.mx4_quantize(x, z(4, 144, d=U8)[:, 8:136], sc), lambda: eff.mx4_quantize(x, c, z(4, 9, d=U8)[:, :8]),
        lambda: eff.mx4_quantize(x, z(1, 128, d=U8).expand(4, 128), sc), lambda: eff.mx4_quantize(x, None, sc), lambda: eff.mx4_quantize(x, c, sc.cpu()),
        lambda: eff.mx4_quantize(z(4, 3, 256)[:, :2], z(4, 2, 128, d=U8), z(4, 2, 8, d=U8)), lambda: eff.mx4_quantize(x[0], c[0], sc[0]),
        lambda: eff.mx4_dequantize(c, sc, z(4, 257)), lambda: eff.mx4_dequantize(c, sc, z(4, 128)), lambda: eff.mx4_dequantize(c, sc, y.int()),
        lambda: eff.mx4_dequantize(c, sc, z(1, 256).expand(4, 256)), lambda: eff.mx4_dequantize(None, sc, y), lambda: eff.mx4_dequantize(c[:2], sc, y),
        lambda: eff.mx4_matmul(x, wq, ws, z(4, 7)), lambda: eff.mx4_matmul(x, wq, ws, out.half()), lambda: eff.mx4_matmul(x, wq[:, :64], ws, out),
        lambda: eff.mx4_matmul(x, wq, ws[:5], out), lambda: eff.mx4_matmul(x.float(), wq, ws, out), lambda: eff.mx4_matmul(c, wq, ws, out),
        lambda: eff.mx4_matmul(x, wq, ws, out, x_scales=sc), lambda: eff.mx4_matmul(c, wq, ws, out, x_scales=sc[:3]), lambda: eff.mx4_matmul(c[:, :64], wq, ws, out, x_scales=sc),
        lambda: eff.mx4_matmul(x, wq, ws, out, bias=z(5)), lambda: eff.mx4_matmul(x, wq, ws, out, bias=z(6, d=F32)), lambda: eff.mx4_matmul(x, wq, ws, out, act=7),
        lambda: eff.mx4_matmul(x, wq, ws, out, act="silu"), lambda: eff.mx4_matmul(x, wq, ws, out, act=1.0), lambda: eff.mx4_matmul(x, wq, ws, out, residual=z(4, 5)),
        lambda: eff.mx4_matmul(x, wq, ws, out, pre=z(4, 5)), lambda: eff.mx4_matmul(x, z(5, 128, d=U8), z(5, 8, d=U8), z(4, 2), act=eff.ACT_SWIGLU),
        lambda: eff.mx4_matmul(x, wq.cpu(), ws, out), lambda: eff.mx4_matmul(x, wq, None, out), lambda: eff.mx4_matmul(c, wq, ws, z(4, 6, d=F32), x_scales=sc, bias=z(6, d=F32)),
        lambda: eff.mx4_matmul(c, wq, ws, out, x_scales=sc, residual=out.half()), lambda: eff.mx4_matmul(x, w3, ws3, out), lambda: eff.mx4_matmul(x[0], wq, ws, out),
        lambda: eff.mx4_matmul(x, z(6, 136, d=U8)[:, :128], ws, out), lambda: eff.mx4_matmul(x, z(6, 129, d=U8).view(-1)[1:769].view(6, 128), ws, out),
        lambda: eff.grouped_mx4_matmul(x, wq, ws, off, out), lambda: eff.grouped_mx4_matmul(x, w3, ws3, off[:2], out), lambda: eff.grouped_mx4_matmul(x, w3, ws3, off.long(), out),
        lambda: eff.grouped_mx4_matmul(x, w3, ws3, None, out), lambda: eff.grouped_mx4_matmul(x, w3, ws3[:1], off, out), lambda: eff.grouped_mx4_matmul(x, w3, ws3, off, out, bias=z(6)),
        lambda: eff.grouped_mx4_matmul(x, z(0, 6, 128, d=U8), z(0, 6, 8, d=U8), z(1, d=I32), out),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(eff.EffError) as ei:
            call()
        assert ei.value.code == eff.EFF_EINVAL, i
