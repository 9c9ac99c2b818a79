"""The operators without an engine in a row, as a model uses them: a mixture layer with its shared expert and its
training step, and a predictor whose ids the decode step takes as its speculative request.  Every stage is held
against 64 bits of its definition on the inputs that it really had."""
import numpy as np
import pytest
import torch

import synth
from synth.configs import TINY
from tests import ops_ref as R
from tests.helpers import PinnedPool, assert_close_bf16, make_engine, oracle_engine

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    return e


def check_product(x, w, y, act=R.NONE, residual=None, off=None, pre=None):
    cpu = [None if t is None else t.cpu() for t in (x, w, residual, off, pre)]
    n = y.shape[1]
    rows = slice(0, x.shape[0]) if off is None else slice(0, int(cpu[3][-1]))
    cpu[0] = cpu[0].clone()
    cpu[0][rows.stop:] = 0
    ry, ye, rz, ze = R.matmul64(cpu[0], cpu[1], None, act, cpu[2], cpu[3], n)
    R.assert_within(y[rows], ry[rows], ye[rows], "product")
    if pre is not None:
        R.assert_within(pre[rows], rz[rows], ze[rows], "pre")


def check_grads(dy, x, w, pre, act, off, dx, dw):
    dy, x, w, pre, off = [None if t is None else t.cpu() for t in (dy, x, w, pre, off)]
    m, nw = x.shape[0], w.shape[-2]
    dyd, xd, wd = dy.double(), x.double(), w.double()
    dz, mag = (dyd, dyd.abs()) if act == R.NONE else R.dz64(dyd, pre.double(), act)
    func = R.FUNC * mag if act else torch.zeros_like(dz)
    ze = func + (R.half_ulp(BF) if act else 0.0) * (dz.abs() + func)
    for e, rows in R.groups_of(off, m):
        we = wd if e is None else wd[e]
        z, err, xr = dz[rows], ze[rows], xd[rows]
        R.assert_within(dx[rows], z @ we, err @ we.abs() + (nw + 8) * R.STEP * ((z.abs() + err) @ we.abs()), "dx")
        R.assert_within(dw if e is None else dw[e], z.t() @ xr,
                        err.t() @ xr.abs() + (len(z) + 8) * R.STEP * ((z.abs() + err).t() @ xr.abs()), "dw")


@pytest.mark.parametrize("T,H,I,E,K", [(1, 64, 32, 4, 2), (37, 128, 72, 8, 3), (150, 264, 96, 40, 6)])
def test_training_step_of_a_mixture_layer(eff, T, H, I, E, K):
    g = torch.Generator().manual_seed(T)
    rnd = lambda *s, scale=1.0: (torch.randn(s, generator=g) * scale).to(BF).cuda()  # noqa: E731
    new = lambda *s, dtype=BF: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    i32 = torch.int32
    x, wr = rnd(T, H), rnd(E, H, scale=H ** -0.5)
    w1, w2 = rnd(E, 2 * I, H, scale=H ** -0.5), rnd(E, H, I, scale=I ** -0.5)
    s1, s2 = rnd(2 * I, H, scale=H ** -0.5), rnd(H, I, scale=I ** -0.5)
    P = T * K
    # forward: router logits, routing (one pair left to the host), shared expert, experts, combine
    logits = new(T, E, dtype=F32)
    eff.matmul(x, wr, logits)
    top, ids = torch.topk(logits, K, dim=1)
    w, ids = torch.softmax(top, 1), ids.to(i32)
    ids[T // 2, 0] = -1
    off, order, pos = new(E + 1, dtype=i32), new(P, dtype=i32), new(T, K, dtype=i32)
    eff.sort_tokens(ids, off, order, pos)
    xs, a, z1, ys = new(P, H), new(P, I), new(P, 2 * I), new(P, H)
    eff.dispatch_tokens(x, pos, xs)
    eff.grouped_matmul(xs, w1, off, a, act=eff.ACT_SWIGLU, pre=z1)
    eff.grouped_matmul(a, w2, off, ys)
    sa, sz, base, out = new(T, I), new(T, 2 * I), new(T, H), new(T, H)
    eff.matmul(x, s1, sa, act=eff.ACT_SWIGLU, pre=sz)
    eff.matmul(sa, s2, base, residual=x)
    eff.combine_tokens(ys, pos, w, out, residual=base)
    # backward
    dout = rnd(T, H)
    dys, dw, da, dxs, dx = new(P, H), new(T, K, dtype=F32), new(P, I), new(P, H), new(T, H)
    dw1, dw2, ds1, ds2, dsa, dxf = new(E, 2 * I, H), new(E, H, I), new(2 * I, H), new(H, I), new(T, I), new(T, H)
    eff.combine_tokens_backward(dout, ys, pos, w, dys, dw)
    eff.grouped_matmul_backward(dys, a, w2, off, dx=da, dw=dw2)
    eff.grouped_matmul_backward(da, xs, w1, off, dx=dxs, dw=dw1, act=eff.ACT_SWIGLU, pre=z1)
    eff.dispatch_tokens_backward(dxs, pos, dx)
    eff.matmul_backward(dout, sa, s2, dx=dsa, dw=ds2)
    eff.matmul_backward(dsa, x, s1, dx=dxf, dw=ds1, act=eff.ACT_SWIGLU, pre=sz)
    torch.cuda.synchronize()

    ro, rr, rp = R.sort_ref(ids.cpu(), E)
    assert torch.equal(off.cpu(), ro) and torch.equal(order.cpu(), rr) and torch.equal(pos.cpu(), rp)
    n = int(ro[-1])
    check_product(x, wr, logits)
    assert torch.equal(xs[:n], x[(rr[:n] // K).long().cuda()])
    check_product(xs, w1, a, act=R.SWIGLU, off=off, pre=z1)
    check_product(a, w2, ys, off=off)
    check_product(x, s1, sa, act=R.SWIGLU, pre=sz)
    check_product(sa, s2, base, residual=x)
    wd, yd, pd = w.cpu().double(), ys.cpu().double(), rp.long()
    ref, mag = base.cpu().double(), base.cpu().double().abs()
    rdx, rmag = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    dd, dxd = dout.cpu().double(), dxs.cpu().double()
    rdw, rdwm = torch.zeros(T, K, dtype=torch.float64), torch.zeros(T, K, dtype=torch.float64)
    rdys = torch.zeros(n, H, dtype=torch.float64)
    for k in range(K):
        at = (pd[:, k] >= 0).nonzero().reshape(-1)
        p = pd[at, k]
        ref[at] += wd[at, k, None] * yd[p]
        mag[at] += (wd[at, k, None] * yd[p]).abs()
        rdx[at] += dxd[p]
        rmag[at] += dxd[p].abs()
        rdw[at, k], rdwm[at, k] = (dd[at] * yd[p]).sum(1), (dd[at] * yd[p]).abs().sum(1)
        rdys[p] = wd[at, k, None] * dd[at]
    R.assert_within(out, ref, (K + 2) * 2.0 ** -24 * mag, "combine")
    R.assert_within(dys[:n], rdys, 2.0 ** -24 * rdys.abs(), "dys")
    R.assert_within(dw, rdw, (H + 8) * 2.0 ** -23 * rdwm, "dw")
    check_grads(dys[:n], a[:n], w2, None, R.NONE, off, da, dw2)
    check_grads(da[:n], xs[:n], w1, z1[:n], R.SWIGLU, off, dxs, dw1)
    R.assert_within(dx, rdx, (K + 2) * 2.0 ** -24 * rmag, "dispatch backward")
    check_grads(dout, sa, s2, None, R.NONE, None, dsa, ds2)
    check_grads(dsa, x, s1, sz, R.SWIGLU, None, dxf, ds1)


def test_predictor_drives_the_speculative_request(eff):
    """fc1 -> gelu -> fc2 + a linear residual gives fp32 logits of the next layer's experts; their top-K, by the engine's
    own router, is the decode step's speculative request.  Ids, slots, counts and outputs as the oracle's."""
    W = TINY
    pool = PinnedPool(eff, W.seed, W.L, W.E, W.H, W.I, W.fmt)
    try:
        eng = make_engine(eff, pool, W.K, 6, 1, 65536)
        orc = oracle_engine(pool, W.K, 6, 65536)
        from oracle.router import topk_softmax
        g = torch.Generator().manual_seed(1)
        fc1, b1 = (torch.randn(128, W.H, generator=g) * W.H ** -0.5).to(BF).cuda(), torch.randn(128, generator=g).to(BF).cuda()
        fc2, lin = (torch.randn(W.E, 128, generator=g) * 0.1).to(BF).cuda(), (torch.randn(W.E, W.H, generator=g) * 0.1).to(BF).cuda()
        h, res = torch.empty(1, 128, dtype=BF, device="cuda"), torch.empty(1, W.E, dtype=BF, device="cuda")
        logits = torch.empty(1, W.E, dtype=F32, device="cuda")
        ids, w = torch.empty(1, W.K, dtype=torch.int32, device="cuda"), torch.empty(1, W.K, dtype=F32, device="cuda")
        side = torch.cuda.Stream()
        spec = 0
        for t in range(6):
            for l in range(W.L):
                xb = synth.activations(W.seed, l, t, 1, W.H)
                wrb = synth.router_weights(W.seed, l, W.E, W.H)
                x = torch.from_numpy(xb.view(np.int16)).cuda()
                xf = x.view(BF)
                eff.matmul(xf, fc1, h, bias=b1, act=eff.ACT_GELU)
                eff.matmul(xf, lin, res)
                eff.matmul(h, fc2, logits, residual=res)
                eng.route_logits(logits, ids, w)
                out = torch.empty((1, W.H), dtype=torch.int16, device="cuda")
                eng.decode_layer(l, x, out, w_router=torch.from_numpy(wrb.view(np.int16)).cuda(), spec_ids=ids if l + 1 < W.L else None,
                                 side=side)
                torch.cuda.synchronize()
                R.assert_within(h, *R.matmul64(xf.cpu(), fc1.cpu(), b1.cpu(), R.GELU, None, None, 128)[:2], "fc1")
                R.assert_within(logits, *R.matmul64(h.cpu(), fc2.cpu(), None, R.NONE, res.cpu(), None, W.E)[:2], "fc2")
                want = topk_softmax(logits.cpu().numpy(), W.K)[0]
                assert np.array_equal(ids.cpu().numpy(), want)
                r = orc.decode_layer(l, xb, router_bits=wrb, spec_next=want if l + 1 < W.L else None)
                got = eng.last_layer_arrays(1)
                assert list(got["ids"]) == list(r["ids"].reshape(-1)) and list(got["slots"]) == r["slots"]
                if r["spec"] is not None:
                    assert list(got["counts"][3:5]) == [r["spec"].m, r["spec"].q]
                    spec += r["spec"].q
                assert_close_bf16(out.cpu().numpy().view(np.uint16), r["out_bits"], what="decode")
        assert spec > 0
        eng.close()
    finally:
        pool.free()
