"""Tokens sorted by expert and back, and their gradients, against the definitions."""
import pytest
import torch

from tests import ops_ref as R

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    return e


def routing(T, K, E, seed=0, masked=0.0, skew=0.0):
    g = torch.Generator().manual_seed(seed + 7 * T + 13 * K + E)
    p = torch.arange(1, E + 1).float() ** -skew
    ids = torch.multinomial(p.expand(T, E), K, generator=g).to(torch.int32) if T else torch.zeros((0, K), dtype=torch.int32)
    ids[torch.rand((T, K), generator=g) < masked] = -1
    return ids


def do_sort(eff, ids, E):
    d = ids.cuda()
    out = [torch.full((E + 1,), 77, dtype=torch.int32, device="cuda"), torch.full((ids.numel(),), 77, dtype=torch.int32, device="cuda"),
           torch.full_like(d, 77)]
    eff.sort_tokens(d, *out)
    return out


@pytest.mark.parametrize("T,K,E,masked,skew", [
    (0, 2, 8, 0, 0), (1, 1, 1, 0, 0), (1, 8, 256, 0, 0), (16, 10, 512, 0, 1.2), (7, 3, 5, 0.5, 0), (64, 1, 64, 0, 0),
    (65, 2, 3, 0.1, 1), (500, 8, 256, 0.1, 1), (1024, 8, 256, 0, 0), (1025, 8, 256, 0.3, 1), (2048, 6, 256, 0, 0.5),
    (5000, 10, 512, 0.1, 1.2), (333, 32, 4096, 0, 0), (3000, 4, 4096, 0.2, 0.5), (100, 4, 2049, 0, 0), (9000, 2, 2, 0, 0),
    (8193, 1, 1, 0.5, 0), (300, 5, 1500, 1.0, 0), (5000, 5, 3000, 1.0, 0)])
def test_sort(eff, T, K, E, masked, skew):
    ids = routing(T, K, E, masked=masked, skew=skew)
    got = do_sort(eff, ids, E)
    for a, b, name in zip(got, R.sort_ref(ids, E), ("offsets", "order", "pos")):
        assert torch.equal(a.cpu(), b), name


@pytest.mark.parametrize("n", [100, 20000])
def test_sort_of_any_ids(eff, n):
    """Ids that no router gives: outside the experts on both sides, and all the same one."""
    E = 37
    g = torch.Generator().manual_seed(n)
    ids = torch.randint(-50, 90, (n,), generator=g, dtype=torch.int32)
    ids[::7], ids[3::11] = -2147483648, 2147483647
    for v in (ids, torch.full((n,), 36, dtype=torch.int32), torch.full((n,), 37, dtype=torch.int32)):
        for a, b in zip(do_sort(eff, v, E), R.sort_ref(v, E)):
            assert torch.equal(a.cpu(), b)


def test_sort_of_many_pairs(eff):
    """More pairs than the definition's loop is run for: against a stable sort."""
    E, n = 100, 1 << 21
    ids = torch.randint(-1, E + 1, (n,), dtype=torch.int32, generator=torch.Generator().manual_seed(1))
    offsets, order, pos = [t.cpu().long() for t in do_sort(eff, ids, E)]
    key = torch.where((ids >= 0) & (ids < E), ids, E).long()
    want = torch.sort(key, stable=True)[1]
    cnt = int((key < E).sum())
    assert offsets[-1] == cnt and torch.equal(order[:cnt], want[:cnt]) and (order[cnt:] == -1).all()
    assert torch.equal(offsets, torch.cat([torch.zeros(1, dtype=torch.int64), torch.bincount(key, minlength=E + 1)[:E].cumsum(0)]))
    assert torch.equal(pos[order[:cnt]], torch.arange(cnt)) and (pos[key == E] == -1).all()


ROWS = [(1, 1, 1, 4), (1, 8, 64, 256), (16, 10, 2560, 512), (33, 3, 100, 9), (40, 2, 77, 5), (5, 32, 520, 64), (130, 6, 2056, 16),
        (64, 4, 4096, 8), (9, 7, 4100, 12)]


def pad_rows(t, pad):
    if not pad:
        return t.cuda()
    big = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    big[:, :t.shape[1]] = t.cuda()
    return big[:, :t.shape[1]]


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T,K,H,E", ROWS)
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_dispatch_and_back(eff, T, K, H, E, dtype, pad):
    ids = routing(T, K, E, masked=0.2)
    ids[T // 2] = -1                       # a token without any pair
    _, order, pos = R.sort_ref(ids, E)
    g = torch.Generator().manual_seed(H)
    x = torch.randn(T, H, generator=g).to(dtype)
    n = T * K
    xs = pad_rows(torch.full((n, H), 7.0, dtype=dtype), pad)
    eff.dispatch_tokens(pad_rows(x, pad), pos.cuda(), xs)
    want = torch.full((n, H), 7.0, dtype=dtype)
    for place, p in enumerate(order.tolist()):
        if p >= 0:
            want[place] = x[p // K]
    assert torch.equal(xs.cpu(), want)
    # gradient: the sum of the rows of a token's pairs; rows of no pair hold NaN and are not read
    d = torch.randn(n, H, generator=g).to(dtype)
    d[order < 0] = float("nan")
    dx = pad_rows(torch.full((T, H), 7.0, dtype=dtype), pad)
    eff.dispatch_tokens_backward(pad_rows(d, pad), pos.cuda(), dx)
    ref, mag = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for place, p in enumerate(order.tolist()):
        if p >= 0:
            ref[p // K] += d[place].double()
            mag[p // K] += d[place].double().abs()
    R.assert_within(dx, ref, (K + 2) * 2.0 ** -24 * mag, "dispatch backward")
    if pad:
        assert torch.isnan(dx.as_strided((T, pad), (dx.stride(0), 1), H)).all()


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T,K,H,E", ROWS)
@pytest.mark.parametrize("pad,residual", [(0, True), (0, False), (1, True), (8, False)])
def test_combine_and_its_gradients(eff, T, K, H, E, dtype, pad, residual):
    ids = routing(T, K, E, masked=0.2)
    ids[T // 2] = -1
    _, order, pos = R.sort_ref(ids, E)
    g = torch.Generator().manual_seed(H + 1)
    n = T * K
    ys, r, dout = (torch.randn(s, H, generator=g).to(dtype) for s in (n, T, T))
    w = torch.softmax(torch.randn(T, K, generator=g), 1)
    ys[order < 0] = float("nan")           # rows of no pair are not read
    w[pos < 0] = float("inf")              # weights of unrouted pairs are not used
    out = pad_rows(torch.full((T, H), 7.0, dtype=dtype), pad)
    eff.combine_tokens(pad_rows(ys, pad), pos.cuda(), w.cuda(), out, residual=pad_rows(r, pad) if residual else None)
    dys, dw = pad_rows(torch.full((n, H), 7.0, dtype=dtype), pad), torch.full((T, K), 7.0, device="cuda")
    eff.combine_tokens_backward(pad_rows(dout, pad), pad_rows(ys, pad), pos.cuda(), w.cuda(), dys, dw)
    ref = r.double() if residual else torch.zeros(T, H, dtype=torch.float64)
    mag = ref.abs()
    rys = torch.full((n, H), 7.0, dtype=torch.float64)
    rdw, dwmag = torch.zeros(T, K, dtype=torch.float64), torch.zeros(T, K, dtype=torch.float64)
    for t in range(T):
        for k in range(K):
            p = int(pos[t, k])
            if p < 0:
                continue
            v, wk = ys[p].double(), float(w[t, k])
            ref[t] = ref[t] + wk * v
            mag[t] = mag[t] + (wk * v).abs()
            rys[p] = wk * dout[t].double()
            rdw[t, k] = (dout[t].double() * v).sum()
            dwmag[t, k] = (dout[t].double() * v).abs().sum()
    R.assert_within(out, ref, (K + 2) * 2.0 ** -24 * mag, "combine")
    R.assert_within(dys, rys, 2.0 ** -24 * rys.abs(), "dys")
    R.assert_within(dw, rdw, (H + 8) * 2.0 ** -23 * dwmag, "dw")
    only = pad_rows(torch.full((n, H), 7.0, dtype=dtype), pad)
    eff.combine_tokens_backward(pad_rows(dout, pad), pad_rows(ys, pad), pos.cuda(), w.cuda(), only)
    assert torch.equal(only, dys)


def test_combine_gradients_against_differences(eff):
    """The combine is linear in ys and in w: differences with h = 1 are its gradients exactly."""
    T, K, H = 3, 2, 8
    g = torch.Generator().manual_seed(2)
    ids = torch.tensor([[1, 0], [-1, 1], [0, 1]], dtype=torch.int32)
    _, order, pos = R.sort_ref(ids, 2)
    ys, c = (torch.randint(-4, 5, (s, H), generator=g).float() for s in (T * K, T))
    w = torch.randint(1, 5, (T, K), generator=g).float() / 4
    dys, dw = torch.zeros(T * K, H, device="cuda"), torch.zeros(T, K, device="cuda")
    eff.combine_tokens_backward(c.cuda(), ys.cuda(), pos.cuda(), w.cuda(), dys, dw)

    def loss(ys, w):
        out = torch.empty(T, H, device="cuda")
        eff.combine_tokens(ys.cuda(), pos.cuda(), w.cuda(), out)
        return float((out.cpu() * c).sum())

    base = loss(ys, w)
    for v, got in ((ys, dys), (w, dw)):
        for j in range(v.numel()):
            up = v.clone()
            up.view(-1)[j] += 1
            assert loss(up if v is ys else ys, up if v is w else w) - base == float(got.view(-1)[j]), j


def test_places_outside_the_rows(eff):
    """Places that sort_tokens would not give are skipped like unrouted pairs: nothing is read or written outside."""
    T, K, H, rows = 4, 3, 64, 5
    pos = torch.tensor([[0, 5, -1], [4, 100, -7], [2147483647, 2, -2147483648], [9, 8, 7]], dtype=torch.int32, device="cuda")
    ok = (pos >= 0) & (pos < rows)
    buf = torch.full((rows + 8, H), 7.0, dtype=BF, device="cuda")
    x = torch.randn(T, H, device="cuda").to(BF)
    eff.dispatch_tokens(x, pos, buf[4:4 + rows])
    assert (buf[:4] == 7).all() and (buf[4 + rows:] == 7).all()
    assert torch.equal(buf[4], x[0]) and torch.equal(buf[8], x[1]) and torch.equal(buf[6], x[2])
    w = torch.ones(T, K, device="cuda")
    out = torch.empty(T, H, dtype=BF, device="cuda")
    eff.combine_tokens(buf[4:4 + rows], pos, w, out)
    assert torch.equal(out[:3], x[:3]) and (out[3] == 0).all()
    dys, dw = torch.full_like(buf, 7.0), torch.empty(T, K, device="cuda")
    eff.combine_tokens_backward(x, buf[4:4 + rows], pos, w, dys[4:4 + rows], dw)
    assert (dys[:4] == 7).all() and (dys[4 + rows:] == 7).all() and (dw[~ok] == 0).all() and (dw[ok] != 0).all()


def test_in_place_and_broadcast_residual(eff):
    T, K, H = 6, 2, 40
    pos = torch.arange(T * K, dtype=torch.int32, device="cuda").view(T, K)
    ys, r = torch.randn(T * K, H, device="cuda"), torch.randn(T, H, device="cuda")
    w = torch.rand(T, K, device="cuda")
    a, b = torch.empty_like(r), r.clone()
    eff.combine_tokens(ys, pos, w, a, residual=r)
    eff.combine_tokens(ys, pos, w, b, residual=b)
    assert torch.equal(a, b)
    eff.combine_tokens(ys, pos, w, b, residual=r[:1].expand(T, H))
    eff.combine_tokens(ys, pos, w, a, residual=r[:1].repeat(T, 1))
    assert torch.equal(a, b)


def test_many_tokens_and_far_rows(eff):
    """More tokens than one grid dimension holds, rows beyond 2^31 elements from the first."""
    T, K, H = 70000, 1, 8
    pos = torch.randperm(T, dtype=torch.int32, device="cuda").view(T, K)
    ld = 40960
    xs = torch.empty(T * ld, dtype=BF, device="cuda").as_strided((T, H), (ld, 1))
    x = torch.randn(T, H, device="cuda").to(BF)
    eff.dispatch_tokens(x, pos, xs)
    assert torch.equal(xs[pos[:, 0].long()], x)
    w = torch.ones(T, K, device="cuda")
    out = torch.empty_like(x)
    eff.combine_tokens(xs, pos, w, out)
    assert torch.equal(out, x)
    eff.dispatch_tokens_backward(xs, pos, out)
    assert torch.equal(out, x)
    dw = torch.empty(T, K, device="cuda")
    dys = torch.empty(T * ld, dtype=BF, device="cuda").as_strided((T, H), (ld, 1))
    eff.combine_tokens_backward(x, xs, pos, w, dys, dw)
    assert torch.equal(dys[pos[:, 0].long()], x)
    R.assert_within(dw[:, 0], (x.double() ** 2).sum(1).cpu(), (H + 8) * 2.0 ** -23 * (x.double() ** 2).sum(1).cpu(), "dw")
    del xs, dys
    torch.cuda.empty_cache()


def test_streams_and_graphs(eff):
    """Sort, dispatch and combine in a graph, replayed on new routings with eager work between, and on two streams."""
    for T, K, E, H in ((16, 10, 512, 256), (2000, 6, 256, 64)):
        ids = routing(T, K, E, masked=0.1).cuda()
        x = torch.randn(T, H, device="cuda").to(BF)
        w = torch.rand(T, K, device="cuda")

        def chain(stream=None):
            off, order, pos = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((E + 1,), (T * K,), (T, K)))
            xs, out, dys, dw = (torch.zeros(s, H, dtype=BF, device="cuda") for s in (T * K, T, T * K, T))
            dw = torch.zeros(T, K, device="cuda")
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
            eff.sort_tokens(ids, off, order, pos, stream=stream)
            eff.dispatch_tokens(x, pos, xs, stream=stream)
            eff.combine_tokens(xs, pos, w, out, residual=x, stream=stream)
            eff.combine_tokens_backward(out, xs, pos, w, dys, dw, stream=stream)
            return off, order, pos, xs, out, dys, dw

        want = chain()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        both = [chain(streams[i % 2]) for i in range(4)]
        torch.cuda.synchronize()
        for got in both:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = chain()
        for i in range(4):
            ids.copy_(routing(T, K, E, seed=i + 1, masked=0.2))
            x.copy_(torch.randn(T, H).to(BF))
            graph.replay()
            torch.cuda.synchronize()
            got = [o.clone() for o in outs]
            for a, b in zip(got, chain()):
                assert torch.equal(a, b), i
