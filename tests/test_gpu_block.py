"""Layer norm, the router's losses and the 4-bit products in a row with the operators around them, as a block is trained and
served; captured, on other streams, from two threads.  Every stage is held against 64 bits of its definition on the inputs
that it really had."""
import threading

import pytest
import torch

from tests import block_ref as B
from tests import ops_ref as R
from tests.test_gpu_moe_layer import check_grads

pytestmark = pytest.mark.gpu
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    return e


class Block:
    """A block's parameters and buffers, and its training step in the library's calls."""

    def __init__(self, eff, T, H, I, E, K, seed=0):
        self.eff, self.T, self.H, self.I, self.E, self.K = eff, T, H, I, E, K
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s, scale=1.0: (torch.randn(s, generator=g) * scale).to(BF).cuda()  # noqa: E731
        new = lambda *s, dtype=BF: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        P = T * K
        self.x, self.dout = rnd(T, H), rnd(T, H)
        self.nw, self.nb = (1 + 0.2 * torch.randn(H, generator=g)).cuda(), (0.1 * torch.randn(H, generator=g)).cuda()
        self.wr, self.w1, self.w2 = rnd(E, H, scale=H ** -0.5), rnd(E, 2 * I, H, scale=H ** -0.5), rnd(E, H, I, scale=I ** -0.5)
        self.mask = (torch.rand(T, generator=g) > 0.2).cuda()
        self.dlosses = torch.tensor([1e-2, 1e-3], device="cuda")
        code = lambda *s: [new(*s[:-1], b, dtype=U8) for b in eff.mx4_row_bytes(s[-1])]  # noqa: E731
        self.w1q, self.w2q, self.xq, self.aq = code(E, 2 * I, H), code(E, H, I), code(P, H), code(P, I)
        self.y, self.mean, self.rstd = new(T, H), new(T, dtype=F32), new(T, dtype=F32)
        self.logits, self.lse, self.losses, self.counts = new(T, E, dtype=F32), new(T, dtype=F32), new(2, dtype=F32), new(E + 1, dtype=I32)
        self.ids, self.w = new(T, K, dtype=I32), new(T, K, dtype=F32)
        self.off, self.order, self.pos = new(E + 1, dtype=I32), new(P, dtype=I32), new(T, K, dtype=I32)
        self.xs, self.z1, self.a, self.ys, self.out = new(P, H), new(P, 2 * I), new(P, I), new(P, H), new(T, H)
        self.dys, self.dw, self.da, self.dxs, self.dy = new(P, H), new(T, K, dtype=F32), new(P, I), new(P, H), new(T, H)
        self.xd, self.ad, self.w1d, self.w2d = new(P, H), new(P, I), new(E, 2 * I, H), new(E, H, I)
        self.dw1, self.dw2, self.dlogits, self.dwr, self.dyr = new(E, 2 * I, H), new(E, H, I), new(T, E, dtype=F32), new(E, H), new(T, H)
        self.dx, self.dnw, self.dnb = new(T, H), new(H, dtype=F32), new(H, dtype=F32)

    def step(self, stream=None):
        eff, s, st = self.eff, self, dict(stream=stream)
        # forward
        eff.layer_norm(s.x, s.y, weight=s.nw, bias=s.nb, mean=s.mean, rstd=s.rstd, **st)
        eff.matmul(s.y, s.wr, s.logits, **st)
        top, ids = torch.topk(s.logits, s.K, dim=1)
        s.w.copy_(torch.softmax(top, 1))
        s.ids.copy_(torch.where(s.mask[:, None], ids, -1))
        eff.balance_loss(s.logits, s.ids, s.counts, s.lse, s.losses, mask=s.mask, **st)
        eff.sort_tokens(s.ids, s.off, s.order, s.pos, **st)
        eff.mx4_quantize(s.w1, *s.w1q, **st)
        eff.mx4_quantize(s.w2, *s.w2q, **st)
        eff.dispatch_tokens(s.y, s.pos, s.xs, **st)
        eff.mx4_quantize(s.xs, *s.xq, **st)
        eff.grouped_mx4_matmul(s.xq[0], *s.w1q, s.off, s.a, x_scales=s.xq[1], act=eff.ACT_SWIGLU, pre=s.z1, **st)
        eff.mx4_quantize(s.a, *s.aq, **st)
        eff.grouped_mx4_matmul(s.aq[0], *s.w2q, s.off, s.ys, x_scales=s.aq[1], **st)
        eff.combine_tokens(s.ys, s.pos, s.w, s.out, residual=s.x, **st)
        # backward, straight through the rounding to 4 bits
        eff.combine_tokens_backward(s.dout, s.ys, s.pos, s.w, s.dys, s.dw, **st)
        for q, d in ((s.xq, s.xd), (s.aq, s.ad), (s.w1q, s.w1d), (s.w2q, s.w2d)):
            eff.mx4_dequantize(*q, d, **st)
        eff.grouped_matmul_backward(s.dys, s.ad, s.w2d, s.off, dx=s.da, dw=s.dw2, **st)
        eff.grouped_matmul_backward(s.da, s.xd, s.w1d, s.off, dx=s.dxs, dw=s.dw1, act=eff.ACT_SWIGLU, pre=s.z1, **st)
        eff.dispatch_tokens_backward(s.dxs, s.pos, s.dy, **st)
        eff.balance_loss_backward(s.logits, s.ids, s.counts, s.lse, s.dlosses, s.dlogits, w=s.w, dw=s.dw, **st)
        eff.matmul_backward(s.dlogits, s.y, s.wr, dx=s.dyr, dw=s.dwr, **st)
        s.dy += s.dyr
        eff.layer_norm_backward(s.dy, s.x, s.mean, s.rstd, dx=s.dx, dw=s.dnw, db=s.dnb, weight=s.nw, residual=s.dout, **st)

    def results(self):
        return [getattr(self, n).clone() for n in ("out", "losses", "counts", "lse", "dx", "dnw", "dnb", "dwr", "dw1", "dw2", "dlogits")]


def check_product(xq, wq, y, off, act, pre=None):
    n = y.shape[1]
    live = int(off[-1])
    xv, wv = B.values(*[t.cpu() for t in xq])[:live], B.values(*[t.cpu() for t in wq])
    off = off.cpu()
    ry, ye, rz, ze = R.matmul64(xv, wv, None, act, None, off, n)
    R.assert_within(y[:live], ry, ye, "product")
    if pre is not None:
        R.assert_within(pre[:live], rz, ze, "pre")


@pytest.mark.parametrize("T,H,I,E,K", [(1, 64, 32, 4, 2), (37, 128, 72, 8, 3), (150, 264, 96, 40, 6), (333, 512, 256, 16, 4)])
def test_training_step_of_a_block(eff, T, H, I, E, K):
    b = Block(eff, T, H, I, E, K, T)
    b.mask[0] = True
    b.step()
    torch.cuda.synchronize()
    c = lambda t: t.cpu()  # noqa: E731
    ry, ye, rm, me, rr, re = B.norm64(c(b.x), c(b.nw), c(b.nb), 1e-5)
    R.assert_within(b.y, ry, ye, "norm")
    R.assert_within(b.logits, *R.matmul64(c(b.y), c(b.wr), None, R.NONE, None, None, E)[:2], "logits")
    rl, le, rc, rs, se = B.balance64(c(b.logits), c(b.ids), c(b.mask), E)
    assert torch.equal(c(b.counts).long(), rc)
    R.assert_within(b.losses, rl, le, "losses")
    ro, _, rp = R.sort_ref(c(b.ids), E)
    assert torch.equal(c(b.off), ro) and torch.equal(c(b.pos), rp) and torch.equal(rc[:E], (ro[1:] - ro[:-1]).long())
    n = int(ro[-1])
    for x, q in ((b.w1.view(-1, H), b.w1q), (b.w2.view(-1, I), b.w2q), (b.xs[:n], b.xq), (b.a[:n], b.aq)):
        codes, scales = B.quantise(c(x))
        assert torch.equal(c(q[0]).view(-1, q[0].shape[-1])[:x.shape[0]], B.pack(codes))
        assert torch.equal(c(q[1]).view(-1, q[1].shape[-1])[:x.shape[0]], scales)
    check_product(b.xq, b.w1q, b.a, b.off, R.SWIGLU, b.z1)
    check_product(b.aq, b.w2q, b.ys, b.off, R.NONE)
    for q, d in ((b.xq, b.xd), (b.aq, b.ad), (b.w1q, b.w1d), (b.w2q, b.w2d)):
        assert torch.equal(c(d).double(), B.values(c(q[0]), c(q[1]))[..., :d.shape[-1]])
    check_grads(b.dys[:n], b.ad[:n], b.w2d, None, R.NONE, b.off, b.da, b.dw2)
    check_grads(b.da[:n], b.xd[:n], b.w1d, b.z1[:n], R.SWIGLU, b.off, b.dxs, b.dw1)
    ref, err = B.balance_grad64(c(b.logits), c(b.ids), c(b.counts).long(), c(b.lse), c(b.dlosses), c(b.w), c(b.dw))
    R.assert_within(b.dlogits, ref, err, "dlogits")
    rx, xe, rw, we, rb, be = B.norm_grad64(c(b.dy), c(b.x), c(b.nw), c(b.mean), c(b.rstd), c(b.dout))
    R.assert_within(b.dx, rx, xe, "dx")
    R.assert_within(b.dnw, rw, we, "dw of the norm")
    R.assert_within(b.dnb, rb, be, "db of the norm")


def test_served_from_codes(eff):
    """Tokens quantised once and dispatched as codes (a row of codes moves as 16-bit values) give what quantising the
    dispatched rows gives."""
    b = Block(eff, 50, 256, 64, 12, 4, 3)
    b.step()
    cb, sb = eff.mx4_row_bytes(256)
    tq, ts = torch.empty(50, cb, dtype=U8, device="cuda"), torch.empty(50, sb, dtype=U8, device="cuda")
    eff.mx4_quantize(b.y, tq, ts)
    xq, xsc = torch.zeros(200, cb, dtype=U8, device="cuda"), torch.zeros(200, sb, dtype=U8, device="cuda")
    eff.dispatch_tokens(tq.view(BF), b.pos, xq.view(BF))
    eff.dispatch_tokens(ts.view(BF), b.pos, xsc.view(BF))
    y, y2 = torch.zeros_like(b.a), torch.zeros_like(b.a)
    eff.grouped_mx4_matmul(xq, *b.w1q, b.off, y, x_scales=xsc, act=eff.ACT_SWIGLU)
    eff.grouped_mx4_matmul(b.xs, *b.w1q, b.off, y2, act=eff.ACT_SWIGLU)
    assert torch.equal(y, y2) and torch.equal(y, torch.where(torch.arange(200, device="cuda")[:, None] < b.off[-1], b.a, 0.0))


def test_captured_and_replayed(eff):
    """The step as a graph, replayed on changed inputs with eager work in between: the eager step's bits every time."""
    a, b = Block(eff, 90, 192, 64, 12, 3, 1), Block(eff, 90, 192, 64, 12, 3, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.step()
    for i in range(4):
        gen = torch.Generator().manual_seed(50 + i)
        x, dout = torch.randn(90, 192, generator=gen).to(BF).cuda(), torch.randn(90, 192, generator=gen).to(BF).cuda()
        mask = (torch.rand(90, generator=gen) > 0.3 * i).cuda()
        for t in (a, b):
            t.x.copy_(x), t.dout.copy_(dout), t.mask.copy_(mask)
        g.replay()
        b.step()
        torch.cuda.synchronize()
        for name, u, v in zip(("out", "losses", "counts", "lse", "dx", "dnw", "dnb", "dwr", "dw1", "dw2", "dlogits"), a.results(), b.results()):
            assert torch.equal(u, v), (i, name)


def test_two_graphs_side_by_side(eff):
    """Two captured steps, replayed on two streams at once, keep apart."""
    blocks = [Block(eff, 300, 256, 96, 16, 4, s) for s in (1, 2)]
    want = []
    for b in blocks:
        b.step()
        want.append(b.results())
    torch.cuda.synchronize()
    graphs = []
    for b in blocks:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.step()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for b, w in zip(blocks, want):
            assert all(torch.equal(u, v) for u, v in zip(b.results(), w))


def test_streams(eff):
    """Given as an object, as a handle, or as the current one; two at once."""
    b = Block(eff, 120, 256, 96, 16, 4, 4)
    b.step()
    torch.cuda.synchronize()
    want = b.results()
    side = torch.cuda.Stream()
    for how in (side, side.cuda_stream, None):
        with torch.cuda.stream(side):                       # torch's own operations of the step run there
            for t in (b.dx, b.out, b.dlogits):
                t.zero_()
            b.step(how)
        side.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(b.results(), want))
    blocks, streams = [Block(eff, 120, 256, 96, 16, 4, 4) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for t, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                t.step()
    torch.cuda.synchronize()
    for t in blocks:
        assert all(torch.equal(u, v) for u, v in zip(t.results(), want))


def test_two_threads(eff):
    blocks = [Block(eff, 64, 256, 64, 8, 2, s) for s in (5, 6)]
    want = []
    for b in blocks:
        b.step()
        torch.cuda.synchronize()
        want.append(b.results())
    errors = []

    def work(b, w):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    b.step()
                torch.cuda.current_stream().synchronize()
                assert all(torch.equal(u, v) for u, v in zip(b.results(), w))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(blocks, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_outputs_count_as_written(eff):
    b = Block(eff, 8, 64, 32, 4, 2, 1)
    names = ["y", "mean", "rstd", "counts", "lse", "losses", "xs", "a", "z1", "ys", "dx", "dnw", "dnb", "dlogits", "xd"]
    outs = [getattr(b, n) for n in names] + b.w1q + b.xq
    before = [t._version for t in outs]
    b.step()
    assert all(t._version > v for t, v in zip(outs, before))


def test_stream_of_another_device(eff):
    class Stream:
        cuda_stream, device_index = torch.cuda.current_stream().cuda_stream, 1

    x = torch.ones(4, 64, dtype=BF, device="cuda")
    c, s = [torch.zeros(4, n, dtype=U8, device="cuda") for n in eff.mx4_row_bytes(64)]
    for call in (lambda: eff.layer_norm(x, x.clone(), stream=Stream()), lambda: eff.mx4_quantize(x, c, s, stream=Stream()),
                 lambda: eff.mx4_matmul(x, c, s, torch.empty(4, 4, dtype=BF, device="cuda"), stream=Stream())):
        with pytest.raises(eff.EffError) as ei:
            call()
        assert ei.value.code == eff.EFF_EINVAL
