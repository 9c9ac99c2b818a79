"""Measured cases of the operators around a block's router and its 4-bit experts: layer norm, the router's balance
loss with its counts, microscaled 4-bit floats, and the products of operands held in them.

`run` computes each in its plain form (fp32 torch operations, one rounding at the end) or, where `own`
is true, through the library's entry points.  Rows no pair is sorted into stay as the buffer had them (zeros).
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = ("none", "silu", "gelu", "gelu_tanh", "swiglu")
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK, UNIT = 32, 128        # values that share a scale; rows are padded to whole units


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the norm in front of a block for a decode batch of 16: latency
        {"name": "norm-decode", "kind": "norm", "dtype": "bf16", "wtype": "bf16", "t": 16, "h": 2560, "bias": False},
        # the norm of a long prefill
        {"name": "norm-prefill", "kind": "norm", "dtype": "bf16", "wtype": "f32", "t": 8192, "h": 4096, "bias": True},
        # its backward pass over a training batch, the gradient past the skip connection added
        {"name": "norm-grad", "kind": "norm_grad", "dtype": "bf16", "wtype": "f32", "t": 8192, "h": 4096, "bias": True,
         "residual": True},
        # the router's loss of a prefill chunk, 256 experts, top-6, a tenth of the tokens padding
        {"name": "balance-chunk", "kind": "balance", "dtype": "f32", "t": 2048, "e": 256, "topk": 6, "padded": 0.1,
         "masked": 0.0},
        # its gradient with that of the routing weights over a training batch, 512 experts, top-10, some pairs on the host
        {"name": "balance-grad", "kind": "balance_grad", "dtype": "f32", "t": 16384, "e": 512, "topk": 10, "padded": 0.0,
         "masked": 0.1},
        # a decode batch's activations to 4 bits and back
        {"name": "quantise-decode", "kind": "quantise", "dtype": "bf16", "rows": 16, "k": 2560},
        # the gate and up weights of 16 experts to 4 bits and back, as a training step does with trained weights
        {"name": "quantise-weights", "kind": "quantise", "dtype": "bf16", "rows": 65536, "k": 4096},
        # a shared expert's gate and up products with SwiGLU for a decode batch of 16: weight streaming
        {"name": "product-decode", "kind": "product", "dtype": "bf16", "out": "bf16", "m": 16, "n": 2048, "k": 4096,
         "act": "swiglu", "bias": False, "residual": False, "pre": False},
        # every size odd, fp16, with bias, activation, residual and the saved sums of a training forward
        {"name": "product-odd", "kind": "product", "dtype": "f16", "out": "f16", "m": 333, "n": 515, "k": 2563,
         "act": "silu", "bias": True, "residual": True, "pre": True},
        # a shared expert's gate and up products for a long prefill
        {"name": "product-prefill", "kind": "product", "dtype": "bf16", "out": "bf16", "m": 8192, "n": 4096, "k": 4096,
         "act": "swiglu", "bias": False, "residual": False, "pre": False},
        # 16 tokens' gate and up products over 512 small experts: most experts have one row or none
        {"name": "experts-decode", "kind": "experts", "dtype": "bf16", "t": 16, "topk": 10, "e": 512, "n": 640,
         "k": 2560, "act": "swiglu", "bias": False, "skew": 1.2, "masked": 0.0},
        # a prefill chunk of 2048 tokens over 256 large experts (about 48 rows each)
        {"name": "experts-prefill", "kind": "experts", "dtype": "bf16", "t": 2048, "topk": 6, "e": 256, "n": 2048,
         "k": 4096, "act": "swiglu", "bias": False, "skew": 0.3, "masked": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A matrix width: a multiple of 64 or of 8 mostly, now and then odd."""
    v, r = _log(rng, lo, hi), rng.random()
    return max(64, v // 64 * 64) if r < 0.5 else max(8, v // 8 * 8) if r < 0.75 else v | 1


def draw(rng):
    kind = rng.choice(["norm", "norm_grad", "balance", "balance_grad", "quantise", "product", "product", "experts", "experts"])
    c = {"kind": kind, "dtype": rng.choice(["bf16", "bf16", "f16"])}
    if kind in ("norm", "norm_grad"):
        c["dtype"] = rng.choice(["bf16", "bf16", "f16", "f32"])
        c.update(wtype=rng.choice([c["dtype"], "f32"]), t=_log(rng, 1, 8192), h=_width(rng, 64, 4096), bias=rng.random() < 0.5)
        if kind == "norm_grad":
            c["residual"] = rng.random() < 0.5
    elif kind in ("balance", "balance_grad"):
        e = _log(rng, 4, 512)
        c["dtype"] = rng.choice(["f32", "f32", "bf16"])
        c.update(t=_log(rng, 1, 16384), e=e, topk=min(e, rng.randint(1, 10)), padded=rng.choice([0.0, 0.1, 0.5]),
                 masked=rng.choice([0.0, 0.1]))
    elif kind == "quantise":
        c["dtype"] = rng.choice(["bf16", "bf16", "f16", "f32"])
        c.update(rows=_log(rng, 1, 32768), k=_width(rng, 64, 4096))
    elif kind == "product":
        c.update(m=_log(rng, 1, 8192), n=_width(rng, 64, 4096), k=_width(rng, 64, 4096), act=rng.choice(ACTS),
                 bias=rng.random() < 0.5, out=c["dtype"] if rng.random() < 0.8 else "f32", residual=rng.random() < 0.5,
                 pre=rng.random() < 0.3)
    else:
        e = _log(rng, 4, 512)
        n, k = _width(rng, 64, 2048), _width(rng, 64, 4096)
        while e * n * k > 256 * 1024 * 2048:
            n, k = max(64, n // 2 // 64 * 64), max(64, k // 2 // 64 * 64)
        c.update(t=_log(rng, 1, 4096), topk=min(e, rng.randint(1, 10)), e=e, n=n, k=k, act=rng.choice(ACTS),
                 bias=rng.random() < 0.5, skew=round(rng.uniform(0.0, 0.5), 2), masked=rng.choice([0.0, 0.1, 0.5]))
    return c


def _rows_of_w(case):
    return case["n"] * (2 if case["act"] == "swiglu" else 1)


def _hit(case):
    """Expected number of experts with a row, for the routing that prepare() draws."""
    p = [(i + 1.0) ** -case["skew"] for i in range(case["e"])]
    s, keep = sum(p), (1.0 - case["masked"]) * case["t"] * case["topk"]
    return sum(-math.expm1(-keep * v / s) for v in p)


def _units(k):
    return (k + UNIT - 1) // UNIT


def work(case):
    kind, b = case["kind"], 4 if case["dtype"] == "f32" else 2
    if kind in ("norm", "norm_grad"):
        t, h, wb = case["t"], case["h"], 4 if case["wtype"] == "f32" else 2
        n = 2 if case["bias"] else 1
        if kind == "norm":
            return {"bytes": 2 * b * t * h + n * wb * h + 8 * t, "flops": 8 * t * h}
        return {"bytes": (4 if case["residual"] else 3) * b * t * h + (1 + n) * wb * h + 8 * t, "flops": 14 * t * h}
    if kind in ("balance", "balance_grad"):
        t, e, pairs = case["t"], case["e"], case["t"] * case["topk"]
        if kind == "balance":
            return {"bytes": b * t * e + 4 * pairs + 4 * t + t + 4 * e, "flops": 6 * t * e}
        return {"bytes": 2 * b * t * e + 12 * pairs + 4 * t + 4 * e, "flops": 8 * t * e}
    if kind == "quantise":
        packed = case["rows"] * _units(case["k"]) * (UNIT // 2 + UNIT // BLOCK)
        return {"bytes": 2 * (b * case["rows"] * case["k"] + packed), "flops": 4 * case["rows"] * case["k"]}
    n, k, nw = case["n"], case["k"], _rows_of_w(case)
    row = _units(k) * (UNIT // 2 + UNIT // BLOCK)
    if kind == "product":
        m, ob = case["m"], 4 if case["out"] == "f32" else b
        return {"bytes": b * m * k + row * nw + (nw * b if case["bias"] else 0) + m * n * (ob + (b if case["residual"] else 0))
                + (m * nw * b if case["pre"] else 0), "flops": 2 * m * nw * k}
    routed = int(case["t"] * case["topk"] * (1.0 - case["masked"]))
    return {"bytes": int(_hit(case) * nw * (row + (b if case["bias"] else 0)) + routed * b * (k + n)), "flops": 2 * routed * nw * k}


# ---------------------------------------------------------------- inputs

def _randn(g, shape, dtype, scale=1.0):
    t = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
    return t.mul_(scale) if scale != 1.0 else t


def _offsets(case, g):
    """offsets [e+1] of the pairs of tokens with distinct experts (popular ones first), a share of the pairs unrouted."""
    t, e, topk = case["t"], case["e"], case["topk"]
    base = -case["skew"] * torch.log(torch.arange(1, e + 1, device="cuda", dtype=torch.float32))
    u = torch.rand((t, e), generator=g, device="cuda").clamp_(1e-20, 1.0 - 1e-7)
    ids = torch.topk(base - torch.log(-torch.log(u)), topk, dim=1)[1]
    drop = torch.rand((t, topk), generator=g, device="cuda") < case["masked"]
    counts = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
    counts.index_add_(0, torch.where(drop, e, ids).reshape(-1), torch.ones(t * topk, dtype=torch.int64, device="cuda"))
    offsets = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(counts[:e], 0)
    return offsets.to(torch.int32)


def _activations(g, shape, dtype):
    """Rows of a residual stream: a mean, a spread that differs by token, and a few columns far larger than the others."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((shape[0], 1), generator=g, device="cuda"))
    x *= torch.where(torch.rand((1, shape[1]), generator=g, device="cuda") < 0.004, 12.0, 1.0)
    return (x + 0.3).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, kind = DT[case["dtype"]], case["kind"]
    s = {"case": case}

    def zeros(*shape, dtype=dt):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    if kind in ("norm", "norm_grad"):
        t, h, wt = case["t"], case["h"], DT[case["wtype"]]
        s["x"] = _activations(g, (t, h), dt)
        s["w"] = (1 + 0.2 * torch.randn(h, generator=g, device="cuda")).to(wt)
        s["b"] = _randn(g, (h,), wt, 0.1) if case["bias"] else None
        if kind == "norm":
            s["y"], s["mean"], s["rstd"] = zeros(t, h), zeros(t, dtype=torch.float32), zeros(t, dtype=torch.float32)
            return s
        x = s["x"].double()
        s["mean"] = x.mean(1).float()
        s["rstd"] = ((x.var(1, unbiased=False) + 1e-5) ** -0.5).float()
        s["dy"] = _randn(g, (t, h), dt)
        s["residual"] = _randn(g, (t, h), dt) if case["residual"] else None
        s["dx"], s["dw"], s["db"] = zeros(t, h), torch.zeros_like(s["w"]), torch.zeros_like(s["w"]) if case["bias"] else None
        return s
    if kind in ("balance", "balance_grad"):
        t, e, topk = case["t"], case["e"], case["topk"]
        popular = 0.7 * torch.randn(e, generator=g, device="cuda")
        s["logits"] = (1.5 * torch.randn((t, e), generator=g, device="cuda") + popular).to(dt)
        top, ids = torch.topk(s["logits"].float(), topk, dim=1)
        drop = torch.rand((t, topk), generator=g, device="cuda") < case["masked"]
        s["ids"] = torch.where(drop, -1, ids).to(torch.int32).contiguous()
        s["mask"] = torch.rand(t, generator=g, device="cuda") >= case["padded"] if case["padded"] else None
        s["counts"] = zeros(e + 1, dtype=torch.int32)
        if kind == "balance":
            s["lse"], s["losses"] = zeros(t, dtype=torch.float32), zeros(2, dtype=torch.float32)
            return s
        live = torch.ones(t, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
        flat = torch.where((s["ids"] >= 0) & live[:, None], s["ids"], e).reshape(-1).long()
        s["counts"][:e] = torch.bincount(flat, minlength=e + 1)[:e].int()
        s["counts"][e] = live.sum().int()
        s["lse"] = torch.where(live, torch.logsumexp(s["logits"].double(), 1), -math.inf).float()
        s["w"] = torch.softmax(top, dim=1).contiguous()
        s["dw"] = torch.where(drop, 0.0, _randn(g, (t, topk), torch.float32, 1e-3)).contiguous()
        s["dlosses"] = torch.tensor([1e-2, 1e-3], device="cuda")
        s["dlogits"] = zeros(t, e)
        return s
    if kind == "quantise":
        rows, k = case["rows"], case["k"]
        s["x"] = _randn(g, (rows, k), dt, 0.02) if rows > 4096 else _activations(g, (rows, k), dt)
        s["codes"] = zeros(rows, _units(k) * UNIT // 2, dtype=torch.uint8)
        s["scales"] = zeros(rows, _units(k) * UNIT // BLOCK, dtype=torch.uint8)
        s["y"] = zeros(rows, k)
        return s
    n, k, nw = case["n"], case["k"], _rows_of_w(case)
    if kind == "experts":
        s["offsets"], m, groups = _offsets(case, g), case["t"] * case["topk"], case["e"]
    else:
        m, groups = case["m"], 1
    s["x"] = _randn(g, (m, k), dt)
    lead = (groups, nw) if kind == "experts" else (nw,)
    s["wq"] = zeros(*lead, _units(k) * UNIT // 2, dtype=torch.uint8)
    s["ws"] = zeros(*lead, _units(k) * UNIT // BLOCK, dtype=torch.uint8)
    for i in range(0, groups, 16):  # quantised weights, as a checkpoint holds them
        part = _randn(g, (min(16, groups - i) * nw, k), torch.float32, k ** -0.5)
        codes, scales = _quantise(part)
        s["wq"].view(groups, nw, -1)[i:i + 16] = _pack(codes).view(-1, nw, s["wq"].shape[-1])
        s["ws"].view(groups, nw, -1)[i:i + 16] = scales.view(-1, nw, s["ws"].shape[-1])
    s["bias"] = _randn(g, (*lead[:-1], nw), dt, 0.5) if case["bias"] else None
    s["residual"] = _randn(g, (m, n), dt) if case.get("residual") else None
    s["y"] = zeros(m, n, dtype=DT[case.get("out", case["dtype"])])
    s["pre"] = zeros(m, nw) if case.get("pre") else None
    return s


# ---------------------------------------------------------------- plain forms

def _power(e):
    """2^e in fp32 of whole numbers e from -126 to 127."""
    return ((e + 127) << 23).view(torch.float32)


def _scale_value(scales):
    """2^(scale - 127), also 2^-127."""
    e = scales.int() - 127
    return _power(torch.clamp(e, min=-126)) * torch.where(e < -126, 0.5, 1.0)


def _quantise(x):
    """Codes (a number each, uint8) and scales of x [m,k] fp32, rows padded with zeros to whole units."""
    m, k = x.shape
    x = torch.nn.functional.pad(x, (0, _units(k) * UNIT - k)).view(m, -1, BLOCK)
    e = torch.frexp(x.abs().amax(2))[1].int() - 3          # floor(log2 of the largest) - 2
    zero = x.abs().amax(2) == 0
    e = torch.where(zero, -127, torch.clamp(e, -127, 127))
    v = x * _power(-e)[..., None]
    a = v.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code += torch.signbit(v).to(torch.uint8) << 3
    return code.view(m, -1), (e + 127).to(torch.uint8)


def _pack(codes):
    """Two codes a byte, the first in the low bits."""
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def _values(codes, scales):
    """What codes (a number each) and scales stand for, fp32."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = table[codes.int()].view(*scales.shape, BLOCK)
    return v.mul_(_scale_value(scales)[..., None]).view(codes.shape)


def _unpack(q):
    return torch.stack([q & 15, q >> 4], dim=-1).view(*q.shape[:-1], -1)


def _act(z, act, n):
    if act == "swiglu":
        gate, up = z[..., :n], z[..., n:]
        return gate / (1 + torch.exp(-gate)) * up
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    return z


def _plain_norm(s):
    case, x = s["case"], s["x"].float()
    dt = DT[case["dtype"]]
    if case["kind"] == "norm":
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5)
        y = d * rstd * s["w"].float()
        if s["b"] is not None:
            y = y + s["b"].float()
        return {"y": y.to(dt), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    g = dy * s["w"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    wt = DT[case["wtype"]]
    return {"dx": dx.to(dt), "dw": (dy * xh).sum(0).to(wt), "db": dy.sum(0).to(wt) if case["bias"] else None}


def _plain_balance(s):
    case, x = s["case"], s["logits"].float()
    e, topk = case["e"], case["topk"]
    if case["kind"] == "balance":
        top = x.amax(1, keepdim=True)
        live = (top[:, 0] > -math.inf) if s["mask"] is None else (top[:, 0] > -math.inf) & s["mask"]
        ex = torch.exp(x - top)
        total = ex.sum(1, keepdim=True)
        lse = torch.where(live, top[:, 0] + torch.log(total[:, 0]), -math.inf)
        p = torch.where(live[:, None], ex / total, 0.0)
        ok = (s["ids"] >= 0) & (s["ids"] < e) & live[:, None]
        counts = torch.zeros(e + 1, dtype=torch.int64, device=x.device)
        counts.index_add_(0, torch.where(ok, s["ids"], e).reshape(-1).long(), torch.ones(ok.numel(), dtype=torch.int64, device=x.device))
        counts[e] = live.sum()
        n = counts[e].clamp(min=1).float()
        f = counts[:e].float() / (n * topk)
        losses = torch.stack([e * (f * p.sum(0)).sum() / n, torch.where(live, lse * lse, 0.0).sum() / n])
        return {"losses": losses, "counts": counts.to(torch.int32), "lse": lse}
    lse = s["lse"]
    live = lse > -math.inf
    p = torch.where(live[:, None], torch.exp(x - lse[:, None]), 0.0)
    n = s["counts"][e].clamp(min=1).float()
    f = s["counts"][:e].float() / (n * topk)
    inner = s["dlosses"][0] * (e / n) * (f - (p * f).sum(1, keepdim=True))
    d = p * (inner + s["dlosses"][1] * (2 / n) * torch.where(live, lse, 0.0)[:, None])
    ok = (s["ids"] >= 0) & live[:, None]
    w, dw = torch.where(ok, s["w"], 0.0), torch.where(ok, s["dw"], 0.0)
    d.scatter_add_(1, s["ids"].clamp(min=0).long(), w * (dw - (w * dw).sum(1, keepdim=True)))
    return {"dlogits": d.to(DT[case["dtype"]])}


def _places(offsets, m):
    """Group and place within its group of every row, which rows belong to one, and the longest group."""
    at = torch.arange(m, device=offsets.device)
    off = offsets.long()
    group = torch.searchsorted(off, at, right=True) - 1
    inside = at < off[-1]
    group = torch.where(inside, group, 0)
    return group, at - off[group], inside, max(1, int((off[1:] - off[:-1]).max()))


def _plain_product(s):
    case = s["case"]
    dt, n = DT[case["dtype"]], case["n"]
    x, w = _values(*_quantise(s["x"].float())), _values(_unpack(s["wq"]), s["ws"])
    if case["kind"] == "experts":
        m = x.shape[0]
        g, p, inside, longest = _places(s["offsets"], m)
        rows = torch.zeros((case["e"], longest, x.shape[1]), dtype=torch.float32, device=x.device)
        rows[g[inside], p[inside]] = x[inside]
        z = rows @ w.transpose(1, 2)
        if s["bias"] is not None:
            z = z + s["bias"].float()[:, None]
        y = torch.zeros((m, n), dtype=torch.float32, device=x.device)
        y[inside] = _act(z, case["act"], n)[g[inside], p[inside]]
        return {"y": y.to(dt)}
    z = x @ w.t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, case["act"], n)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(DT[case["out"]]), "pre": z.to(dt) if case["pre"] else None}


def _plain(s):
    kind = s["case"]["kind"]
    if kind in ("norm", "norm_grad"):
        return _plain_norm(s)
    if kind in ("balance", "balance_grad"):
        return _plain_balance(s)
    if kind == "quantise":
        codes, scales = _quantise(s["x"].float())
        return {"values": _values(codes, scales)[:, :s["case"]["k"]].to(DT[s["case"]["dtype"]]), "scales": scales}
    return _plain_product(s)


# ---------------------------------------------------------------- the library's calls

def _own(s):
    import expert_ffn_serving_amd as eff
    kind = s["case"]["kind"]
    if kind == "norm":
        eff.layer_norm(s["x"], s["y"], weight=s["w"], bias=s["b"], eps=1e-5, mean=s["mean"], rstd=s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if kind == "norm_grad":
        eff.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], dx=s["dx"], dw=s["dw"], db=s["db"], weight=s["w"],
                                residual=s["residual"])
        return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}
    if kind == "balance":
        eff.balance_loss(s["logits"], s["ids"], s["counts"], s["lse"], s["losses"], mask=s["mask"])
        return {"losses": s["losses"], "counts": s["counts"], "lse": s["lse"]}
    if kind == "balance_grad":
        eff.balance_loss_backward(s["logits"], s["ids"], s["counts"], s["lse"], s["dlosses"], s["dlogits"], w=s["w"], dw=s["dw"])
        return {"dlogits": s["dlogits"]}
    if kind == "quantise":
        eff.mx4_quantize(s["x"], s["codes"], s["scales"])
        eff.mx4_dequantize(s["codes"], s["scales"], s["y"])
        return {"values": s["y"], "scales": s["scales"]}
    act = ACTS.index(s["case"]["act"])   # eff.ACT_*: none, silu, gelu, gelu_tanh, swiglu
    if kind == "experts":
        eff.grouped_mx4_matmul(s["x"], s["wq"], s["ws"], s["offsets"], s["y"], bias=s["bias"], act=act)
        return {"y": s["y"]}
    eff.mx4_matmul(s["x"], s["wq"], s["ws"], s["y"], bias=s["bias"], act=act, residual=s["residual"], pre=s["pre"])
    return {"y": s["y"], "pre": s["pre"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _act64(z, act, n):
    if act == "swiglu":
        return z[:, :n] * torch.sigmoid(z[:, :n]) * z[:, n:]
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def _near64(x):
    """The nearest microscaled value of every entry of x [m,k] (k a whole number of blocks), and the blocks' exponents."""
    m, k = x.shape
    b = x.double().view(m, k // BLOCK, BLOCK)
    top = b.abs().amax(2, keepdim=True)
    e = torch.where(top > 0, torch.floor(torch.log2(torch.where(top > 0, top, 1.0))), -math.inf)
    e = torch.where(torch.ldexp(torch.ones_like(top), torch.where(top > 0, e + 1, 0.0)) <= top, e + 1, e)  # log2 just below a power
    e = torch.where((top > 0) & (torch.ldexp(torch.ones_like(top), torch.where(top > 0, e, 0.0)) > top), e - 1, e)
    e = torch.clamp(e - 2, -127, 127)
    v = torch.ldexp(b, -e)
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))   # between neighbours; round() takes ties to the even one
    q = torch.round(a / step) * step
    return torch.ldexp(torch.copysign(q, v), e).view(m, k), e[..., 0]


def _padded64(x):
    return torch.nn.functional.pad(x.double(), (0, _units(x.shape[1]) * UNIT - x.shape[1]))


def _weights64(q, scales):
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=q.device)
    v = torch.empty((q.shape[0], q.shape[1] * 2), dtype=torch.float64, device=q.device)
    v[:, 0::2], v[:, 1::2] = table[(q & 15).long()], table[(q >> 4).long()]
    return v * torch.pow(2.0, scales.double() - 127).repeat_interleave(BLOCK, 1)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        x = s["x"].double()
        y = torch.nn.functional.layer_norm(x, (case["h"],), s["w"].double(), None if s["b"] is None else s["b"].double(), 1e-5)
        return {"y": y, "mean": x.mean(1), "rstd": (x.var(1, unbiased=False) + 1e-5) ** -0.5}
    if kind == "norm_grad":
        # the gradients of <dy, y> at the inputs, for the statistics that were saved
        x, dy, w = s["x"].double(), s["dy"].double(), s["w"].double()
        mean, rstd = s["mean"].double()[:, None], s["rstd"].double()[:, None]
        u = (x - mean) * rstd
        v = dy * w
        h = case["h"]
        dx = (v - (v.sum(1, keepdim=True) + u * (v * u).sum(1, keepdim=True)) / h) * rstd
        return {"dx": dx if s["residual"] is None else dx + s["residual"].double(), "dw": torch.einsum("th,th->h", dy, u),
                "db": dy.sum(0) if case["bias"] else None}
    if kind in ("balance", "balance_grad"):
        e, topk = case["e"], case["topk"]
        grad = kind == "balance_grad"
        live = s["lse"] > -math.inf if grad else torch.ones(case["t"], dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
        with torch.enable_grad():
            x = s["logits"][live].double().requires_grad_(grad)
            n = x.shape[0]
            ids = s["ids"][live].long()
            f = torch.stack([(ids == i).sum() for i in range(e)]).double() / max(1, n * topk)
            lse = torch.logsumexp(x, 1)
            balance = e * (torch.softmax(x, 1).sum(0) * f).sum() / max(1, n)
            z = (lse ** 2).sum() / max(1, n)
            if not grad:
                every = torch.full((case["t"],), -math.inf, dtype=torch.float64, device="cuda")
                every[live] = lse
                return {"losses": torch.stack([balance, z]), "counts": None, "lse": every}
            total = s["dlosses"][0].double() * balance + s["dlosses"][1].double() * z
            out = torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda")
            if n:
                out[live] = torch.autograd.grad(total, x)[0]
        w, dw, rows = s["w"].double(), s["dw"].double(), torch.arange(case["t"], device="cuda")
        at = [(s["ids"][:, k] >= 0) & live for k in range(topk)]
        mean = sum(torch.where(at[k], w[:, k] * dw[:, k], 0.0) for k in range(topk))
        for k in range(topk):
            r = rows[at[k]]
            out[r, s["ids"][r, k].long()] += w[r, k] * (dw[r, k] - mean[r])
        return {"dlogits": out}
    if kind == "quantise":
        v, e = _near64(_padded64(s["x"]))
        return {"values": v[:, :case["k"]], "scales": None}
    act, n = case["act"], case["n"]
    x = _near64(_padded64(s["x"]))[0]
    if kind == "experts":
        off = s["offsets"].tolist()
        parts = [(slice(off[i], off[i + 1]), i) for i in range(case["e"]) if off[i + 1] > off[i]]
    else:
        parts = [(slice(0, case["m"]), None)]
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    for rows, i in parts:
        z = x[rows] @ _weights64(*((s["wq"], s["ws"]) if i is None else (s["wq"][i], s["ws"][i]))).t()
        if s["bias"] is not None:
            z = z + (s["bias"] if i is None else s["bias"][i]).double()
        y[rows] = _act64(z, act, n)
        if s["residual"] is not None:
            y[rows] += s["residual"][rows].double()
    return {"y": y} if kind == "experts" else {"y": y, "pre": z if case["pre"] else None}
