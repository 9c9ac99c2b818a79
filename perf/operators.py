"""Measured cases of the operators around the routed-expert step: dense products with their epilogue,
tokens sorted by expert and back, and the experts' products on the sorted rows.

`run` computes each in its plain form (fp32 torch operations, one rounding at the end) or, where `own`
is true, through the library's entry points.  Rows no pair is sorted into stay as the buffer had them (zeros).
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = ("none", "silu", "gelu", "gelu_tanh", "swiglu")


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the predictor of the next layer's experts, first layer (2560 -> 512, erf-gelu), at one token: latency
        {"name": "product-token", "kind": "product", "dtype": "bf16", "out": "bf16", "m": 1, "n": 512, "k": 2560,
         "act": "gelu", "bias": True, "residual": False, "pre": False},
        # a shared expert's gate and up products with SwiGLU for a decode batch of 16: weight streaming
        {"name": "product-decode-16", "kind": "product", "dtype": "bf16", "out": "bf16", "m": 16, "n": 2048, "k": 4096,
         "act": "swiglu", "bias": False, "residual": False, "pre": False},
        # every size odd, fp16, with bias, activation, residual and the saved sums of a training forward
        {"name": "product-odd", "kind": "product", "dtype": "f16", "out": "f16", "m": 333, "n": 515, "k": 2563,
         "act": "silu", "bias": True, "residual": True, "pre": True},
        # a shared expert's down product with the residual for a long prefill
        {"name": "product-prefill", "kind": "product", "dtype": "bf16", "out": "bf16", "m": 8192, "n": 4096, "k": 2048,
         "act": "none", "bias": False, "residual": True, "pre": False},
        # gradients of a shared expert's gate and up products over a training batch
        {"name": "product-grad", "kind": "product_grad", "dtype": "bf16", "m": 4096, "n": 2048, "k": 4096,
         "act": "swiglu", "bias": True},
        # a decode batch of 16 tokens sorted over 512 experts (top-10) and dispatched
        {"name": "sort-decode", "kind": "sort", "dtype": "bf16", "t": 16, "topk": 10, "e": 512, "h": 2560,
         "skew": 1.2, "masked": 0.0},
        # a long prefill sorted over 256 experts (top-6) and dispatched, some pairs left to the host
        {"name": "sort-prefill", "kind": "sort", "dtype": "bf16", "t": 8192, "topk": 6, "e": 256, "h": 4096,
         "skew": 1.0, "masked": 0.1},
        # the same tokens' expert rows combined with their weights and the residual
        {"name": "combine-prefill", "kind": "combine", "dtype": "bf16", "t": 8192, "topk": 6, "e": 256, "h": 4096,
         "skew": 1.0, "masked": 0.1, "residual": True},
        # its gradients: expert rows and router weights
        {"name": "combine-grad", "kind": "combine_grad", "dtype": "bf16", "t": 4096, "topk": 8, "e": 256, "h": 2048,
         "skew": 1.1, "masked": 0.0},
        # 16 tokens' gate and up products over 512 small experts: most experts have one row or none
        {"name": "experts-decode", "kind": "experts", "dtype": "bf16", "t": 16, "topk": 10, "e": 512, "n": 640,
         "k": 2560, "act": "swiglu", "bias": False, "skew": 1.2, "masked": 0.0},
        # a prefill chunk of 2048 tokens over 256 large experts (about 48 rows each)
        {"name": "experts-prefill", "kind": "experts", "dtype": "bf16", "t": 2048, "topk": 6, "e": 256, "n": 2048,
         "k": 4096, "act": "swiglu", "bias": False, "skew": 0.3, "masked": 0.0},
        # gradients of 256 small experts' gate and up products over a training batch
        {"name": "experts-grad", "kind": "experts_grad", "dtype": "bf16", "t": 4096, "topk": 8, "e": 256, "n": 512,
         "k": 2048, "act": "swiglu", "bias": False, "skew": 0.3, "masked": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A matrix width: a multiple of 64 or of 8 mostly, now and then odd."""
    v, r = _log(rng, lo, hi), rng.random()
    return max(64, v // 64 * 64) if r < 0.5 else max(8, v // 8 * 8) if r < 0.75 else v | 1


def draw(rng):
    kind = rng.choice(["product", "product", "product_grad", "sort", "combine", "combine_grad", "dispatch_grad", "experts",
                       "experts_grad"])
    c = {"kind": kind, "dtype": rng.choice(["bf16", "bf16", "f16"])}
    if kind in ("product", "product_grad"):
        m, n, k = _log(rng, 1, 8192), _width(rng, 64, 4096), _width(rng, 64, 4096)
        c.update(m=m, n=n, k=k, act=rng.choice(ACTS), bias=rng.random() < 0.5)
        if kind == "product":
            c.update(out=c["dtype"] if rng.random() < 0.8 else "f32", residual=rng.random() < 0.5, pre=rng.random() < 0.3)
    elif kind in ("experts", "experts_grad"):
        e = _log(rng, 4, 512)
        n, k = _width(rng, 64, 2048), _width(rng, 64, 4096)
        while e * n * k > 256 * 1024 * 2048:
            n, k = max(64, n // 2 // 64 * 64), max(64, k // 2 // 64 * 64)
        topk = min(e, rng.randint(1, 10))
        t = _log(rng, 1, 4096)
        c.update(t=t, topk=topk, e=e, n=n, k=k, act=rng.choice(ACTS), bias=rng.random() < 0.5,
                 skew=round(rng.uniform(0.0, 0.5), 2), masked=rng.choice([0.0, 0.1, 0.5]))
    else:
        e = _log(rng, 4, 512)
        c["dtype"] = rng.choice(["bf16", "bf16", "f16", "f32"])
        c.update(t=_log(rng, 1, 8192), topk=min(e, rng.randint(1, 10)), e=e, h=_width(rng, 64, 4096),
                 skew=round(rng.uniform(0.0, 1.2), 2), masked=rng.choice([0.0, 0.1, 0.5]))
        if kind == "combine":
            c["residual"] = rng.random() < 0.5
    return c


def _rows_of_w(case):
    return case["n"] * (2 if case["act"] == "swiglu" else 1)


def _hit(case):
    """Expected number of experts with a row, for the routing that prepare() draws."""
    p = [(i + 1.0) ** -case["skew"] for i in range(case["e"])]
    s, keep = sum(p), (1.0 - case["masked"]) * case["t"] * case["topk"]
    return sum(-math.expm1(-keep * v / s) for v in p)


def work(case):
    kind, b = case["kind"], 4 if case["dtype"] == "f32" else 2
    if kind in ("product", "product_grad"):
        m, n, k, nw = case["m"], case["n"], case["k"], _rows_of_w(case)
        nbias = nw * b if case["bias"] else 0
        if kind == "product":
            ob = 4 if case["out"] == "f32" else b
            return {"bytes": b * (m * k + nw * k) + nbias + m * n * (ob + (b if case["residual"] else 0))
                    + (m * nw * b if case["pre"] else 0), "flops": 2 * m * nw * k}
        pre = m * nw if case["act"] != "none" else 0
        return {"bytes": b * (m * n + pre + 2 * m * k + 2 * nw * k) + nbias, "flops": 4 * m * nw * k}
    t, topk, e = case["t"], case["topk"], case["e"]
    pairs = t * topk
    routed = int(pairs * (1.0 - case["masked"]))
    if kind in ("experts", "experts_grad"):
        n, k, nw = case["n"], case["k"], _rows_of_w(case)
        hit = _hit(case)
        if kind == "experts":
            return {"bytes": int(b * (hit * nw * (k + (1 if case["bias"] else 0)) + routed * (k + n))), "flops": 2 * routed * nw * k}
        pre = nw if case["act"] != "none" else 0
        return {"bytes": int(b * (hit * nw * k + e * nw * (k + (1 if case["bias"] else 0)) + routed * (n + pre + 2 * k))),
                "flops": 4 * routed * nw * k}
    h = case["h"]
    if kind == "sort":
        return {"bytes": 4 * (3 * pairs + e + 1) + b * h * (t + routed), "flops": 0}
    if kind == "combine":
        return {"bytes": 8 * pairs + b * h * (routed + t * (2 if case["residual"] else 1)), "flops": 2 * routed * h}
    if kind == "dispatch_grad":
        return {"bytes": 4 * pairs + b * h * (routed + t), "flops": routed * h}
    return {"bytes": 12 * pairs + b * h * (2 * routed + t), "flops": 3 * routed * h}


# ---------------------------------------------------------------- inputs

def _routing(case, g):
    """Distinct experts of every token (popular ones first in the id space), a share of the pairs unrouted (-1)."""
    t, e, topk = case["t"], case["e"], case["topk"]
    base = -case["skew"] * torch.log(torch.arange(1, e + 1, device="cuda", dtype=torch.float32))
    u = torch.rand((t, e), generator=g, device="cuda").clamp_(1e-20, 1.0 - 1e-7)
    logits = base - torch.log(-torch.log(u))
    top, ids = torch.topk(logits, topk, dim=1)
    w = torch.softmax(top, dim=1)
    drop = torch.rand((t, topk), generator=g, device="cuda") < case["masked"]
    return torch.where(drop, -1, ids).to(torch.int32).contiguous(), w.contiguous()


def _sorted(ids, e):
    """offsets [e+1], order [pairs], pos [T,K] of the stable sort by expert; unrouted pairs get no place."""
    flat = ids.reshape(-1).long()
    routed = (flat >= 0) & (flat < e)
    key = torch.where(routed, flat, e)
    order = torch.sort(key, stable=True)[1]
    offsets = torch.zeros(e + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.cumsum(torch.zeros(e + 1, dtype=torch.int64, device=ids.device).index_add_(
        0, key, torch.ones_like(key)), 0)[:e]
    place = torch.arange(flat.numel(), device=ids.device)
    pos = torch.empty_like(flat)
    pos[order] = place
    pos = torch.where(routed, pos, -1)
    order = torch.where(place < offsets[e], order, -1)
    return offsets.to(torch.int32), order.to(torch.int32), pos.to(torch.int32).view(ids.shape)


def _randn(g, shape, dtype, scale=1.0):
    t = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
    return t.mul_(scale) if scale != 1.0 else t


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, kind = DT[case["dtype"]], case["kind"]
    s = {"case": case}

    def zeros(*shape, dtype=dt):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    if kind in ("product", "product_grad", "experts", "experts_grad"):
        n, k, nw = case["n"], case["k"], _rows_of_w(case)
        if kind.startswith("experts"):
            ids, _ = _routing(case, g)
            s["offsets"], m, lead = _sorted(ids, case["e"])[0], ids.numel(), (case["e"],)
        else:
            m, lead = case["m"], ()
        s["x"] = _randn(g, (m, k), dt)
        s["w"] = _randn(g, lead + (nw, k), dt, k ** -0.5)
        s["bias"] = _randn(g, lead + (nw,), dt, 0.5) if case["bias"] else None
        s["residual"] = _randn(g, (m, n), dt) if case.get("residual") else None
        if kind.endswith("_grad"):
            s["dy"] = _randn(g, (m, n), dt)
            s["pre"] = _randn(g, (m, nw), dt) if case["act"] != "none" else None
            s["dx"], s["dw"] = zeros(m, k), zeros(*lead, nw, k)
            s["dbias"] = zeros(*lead, nw) if case["bias"] else None
        else:
            s["y"] = zeros(m, n, dtype=DT[case.get("out", case["dtype"])])
            s["pre"] = zeros(m, nw) if case.get("pre") else None
        return s
    t, h, e = case["t"], case["h"], case["e"]
    s["ids"], s["w"] = _routing(case, g)
    pairs = s["ids"].numel()
    if kind == "sort":
        s["x"] = _randn(g, (t, h), dt)
        s["offsets"] = zeros(e + 1, dtype=torch.int32)
        s["order"], s["pos"] = zeros(pairs, dtype=torch.int32), torch.zeros_like(s["ids"])
        s["xs"] = zeros(pairs, h)
        return s
    s["pos"] = _sorted(s["ids"], e)[2]
    s["rows"] = _randn(g, (pairs, h), dt)     # expert outputs, or the gradient of the dispatched rows
    s["residual"] = _randn(g, (t, h), dt) if case.get("residual") else None
    s["out"] = zeros(t, h)
    if kind == "combine_grad":
        s["dout"] = _randn(g, (t, h), dt)
        s["dys"], s["dw"] = zeros(pairs, h), torch.zeros_like(s["w"])
    return s


# ---------------------------------------------------------------- plain forms

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


def _dz(dy, z, act, n):
    if act == "none":
        return dy
    if act == "swiglu":
        gate, up = z[..., :n], z[..., n:]
        sg = 1 / (1 + torch.exp(-gate))
        return torch.cat([dy * up * sg * (1 + gate * (1 - sg)), dy * gate * sg], dim=-1)
    if act == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return dy * sg * (1 + z * (1 - sg))
    if act == "gelu":
        return dy * (0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5)
    c = (2 / math.pi) ** 0.5
    th = torch.tanh(c * (z + 0.044715 * z * z * z))
    return dy * (0.5 * (1 + th) + 0.5 * z * (1 - th * th) * c * (1 + 3 * 0.044715 * z * z))


def _places(offsets, m):
    """Group and place within its group of every row, which rows belong to one, and the longest group."""
    at = torch.arange(m, device=offsets.device)
    off = offsets.long()
    group = torch.searchsorted(off, at, right=True) - 1
    inside = at < off[-1]
    group = torch.where(inside, group, 0)
    return group, at - off[group], inside, max(1, int((off[1:] - off[:-1]).max()))


def _pad(v, group, place, inside, e, longest):
    p = torch.zeros((e, longest, v.shape[1]), dtype=torch.float32, device=v.device)
    p[group[inside], place[inside]] = v[inside].float()
    return p


def _unpad(p, group, place, inside, like):
    out = torch.zeros(like, dtype=torch.float32, device=p.device)
    out[inside] = p[group[inside], place[inside]]
    return out


def _plain(s):
    case = s["case"]
    kind, dt = case["kind"], DT[case["dtype"]]
    if kind == "product":
        z = s["x"].float() @ s["w"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, case["act"], case["n"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(DT[case["out"]]), "pre": z.to(dt) if case["pre"] else None}
    if kind == "product_grad":
        pre = None if s["pre"] is None else s["pre"].float()
        dz = _dz(s["dy"].float(), pre, case["act"], case["n"])
        return {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.t() @ s["x"].float()).to(dt),
                "dbias": dz.sum(0).to(dt) if case["bias"] else None}
    if kind == "experts":
        e, m = case["e"], s["x"].shape[0]
        g, p, inside, longest = _places(s["offsets"], m)
        z = _pad(s["x"], g, p, inside, e, longest) @ s["w"].float().transpose(1, 2)
        if s["bias"] is not None:
            z = z + s["bias"].float()[:, None]
        return {"y": _unpad(_act(z, case["act"], case["n"]), g, p, inside, (m, case["n"])).to(dt)}
    if kind == "experts_grad":
        e, (m, k) = case["e"], s["x"].shape
        g, p, inside, longest = _places(s["offsets"], m)
        pre = None if s["pre"] is None else s["pre"].float()
        dz = _pad(_dz(s["dy"].float(), pre, case["act"], case["n"]), g, p, inside, e, longest)
        xp = _pad(s["x"], g, p, inside, e, longest)
        return {"dx": _unpad(dz @ s["w"].float(), g, p, inside, (m, k)).to(dt),
                "dw": (dz.transpose(1, 2) @ xp).to(dt), "dbias": dz.sum(1).to(dt) if case["bias"] else None}
    if kind == "sort":
        offsets, order, pos = _sorted(s["ids"], case["e"])
        pairs = pos.numel()
        xs = torch.zeros((pairs + 1, case["h"]), dtype=dt, device=pos.device)
        xs[torch.where(pos >= 0, pos, pairs).reshape(-1).long()] = s["x"].repeat_interleave(case["topk"], 0)
        return {"offsets": offsets, "order": order, "pos": pos, "xs": xs[:pairs]}
    pos = s["pos"].long()
    has = pos >= 0
    rows = s["rows"][pos.clamp(min=0)].float()
    if kind == "combine":
        y = torch.where(has[..., None], s["w"][..., None] * rows, 0.0).sum(1)
        return {"out": (y + s["residual"].float() if s["residual"] is not None else y).to(dt)}
    if kind == "dispatch_grad":
        return {"dx": torch.where(has[..., None], rows, 0.0).sum(1).to(dt)}
    d = s["dout"].float()[:, None]
    dw = torch.where(has, (d * rows).sum(-1), 0.0)
    pairs = pos.numel()
    dys = torch.zeros((pairs + 1, case["h"]), dtype=dt, device=pos.device)
    dys[torch.where(has, pos, pairs).reshape(-1)] = (s["w"][..., None] * d).to(dt).view(pairs, -1)
    return {"dys": dys[:pairs], "dw": dw}


# ---------------------------------------------------------------- the library's calls

def _own(s):
    import expert_ffn_serving_amd as eff
    case = s["case"]
    kind = case["kind"]
    if kind in ("product", "product_grad", "experts", "experts_grad"):
        act = ACTS.index(case["act"])   # eff.ACT_*: none, silu, gelu, gelu_tanh, swiglu
        if kind == "product":
            eff.matmul(s["x"], s["w"], s["y"], bias=s["bias"], act=act, residual=s["residual"], pre=s["pre"])
            return {"y": s["y"], "pre": s["pre"]}
        if kind == "experts":
            eff.grouped_matmul(s["x"], s["w"], s["offsets"], s["y"], bias=s["bias"], act=act)
            return {"y": s["y"]}
        if kind == "product_grad":
            eff.matmul_backward(s["dy"], s["x"], s["w"], dx=s["dx"], dw=s["dw"], dbias=s["dbias"], act=act, pre=s["pre"])
        else:
            eff.grouped_matmul_backward(s["dy"], s["x"], s["w"], s["offsets"], dx=s["dx"], dw=s["dw"], dbias=s["dbias"],
                                        act=act, pre=s["pre"])
        return {"dx": s["dx"], "dw": s["dw"], "dbias": s["dbias"]}
    if kind == "sort":
        eff.sort_tokens(s["ids"], s["offsets"], s["order"], s["pos"])
        eff.dispatch_tokens(s["x"], s["pos"], s["xs"])
        return {"offsets": s["offsets"], "order": s["order"], "pos": s["pos"], "xs": s["xs"]}
    if kind == "combine":
        eff.combine_tokens(s["rows"], s["pos"], s["w"], s["out"], residual=s["residual"])
        return {"out": s["out"]}
    if kind == "dispatch_grad":
        eff.dispatch_tokens_backward(s["rows"], s["pos"], s["out"])
        return {"dx": s["out"]}
    eff.combine_tokens_backward(s["dout"], s["rows"], s["pos"], s["w"], s["dys"], s["dw"])
    return {"dys": s["dys"], "dw": s["dw"]}


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


def _dz64(dy, z, act, n):
    """The gradient at z from autograd of the activation's definition."""
    if act == "none":
        return dy
    with torch.enable_grad():
        z = z.detach().requires_grad_(True)
        return torch.autograd.grad(_act64(z, act, n), z, dy)[0]


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    f = {k: v.double() if v.is_floating_point() else v for k, v in s.items() if isinstance(v, torch.Tensor) and k != "w"}
    if kind in ("product", "product_grad", "experts", "experts_grad"):
        act, n, w = case["act"], case["n"], s["w"]
        if kind.startswith("experts"):
            off = s["offsets"].tolist()
            parts = [(slice(off[i], off[i + 1]), i) for i in range(case["e"]) if off[i + 1] > off[i]]
        else:
            parts = [(slice(0, case["m"]), None)]
        out = {k: torch.zeros(s[k].shape, dtype=torch.float64, device="cuda") for k in ("y", "pre", "dx", "dw", "dbias")
               if s.get(k) is not None and (k != "pre" or not kind.endswith("_grad"))}
        for rows, i in parts:
            we = (w if i is None else w[i]).double()
            x = f["x"][rows]
            if kind.endswith("_grad"):
                dz = _dz64(f["dy"][rows], f["pre"][rows] if "pre" in f else None, act, n)
                out["dx"][rows] = dz @ we
                (out["dw"] if i is None else out["dw"][i]).copy_(dz.t() @ x)
                if "dbias" in out:
                    (out["dbias"] if i is None else out["dbias"][i]).copy_(dz.sum(0))
                continue
            z = x @ we.t()
            if "bias" in f:
                z = z + (f["bias"] if i is None else f["bias"][i])
            y = _act64(z, act, n)
            out["y"][rows] = y + f["residual"][rows] if "residual" in f else y
            if "pre" in out:
                out["pre"][rows] = z
        names = ("dx", "dw", "dbias") if kind.endswith("_grad") else ("y", "pre") if kind == "product" else ("y",)
        return {k: out.get(k) for k in names}
    t, topk = case["t"], case["topk"]
    if kind == "sort":
        pos = _sorted(s["ids"], case["e"])[2].reshape(-1).long()
        xs = torch.zeros((pos.numel(), case["h"]), dtype=torch.float64, device="cuda")
        pairs = torch.nonzero(pos >= 0).reshape(-1)
        xs[pos[pairs]] = f["x"][pairs // topk]
        return {"offsets": None, "order": None, "pos": None, "xs": xs}
    w, pos = s["w"].double(), s["pos"].long()
    y = f["residual"].clone() if "residual" in f else torch.zeros((t, case["h"]), dtype=torch.float64, device="cuda")
    dys = torch.zeros_like(f["rows"])
    dw = torch.zeros_like(w)
    for k in range(topk):
        at = torch.nonzero(pos[:, k] >= 0).reshape(-1)
        rows = f["rows"][pos[at, k]]
        if kind == "combine_grad":
            dys[pos[at, k]] = w[at, k, None] * f["dout"][at]
            dw[at, k] = (f["dout"][at] * rows).sum(1)
        else:
            y[at] += rows if kind == "dispatch_grad" else w[at, k, None] * rows
    if kind == "combine_grad":
        return {"dys": dys, "dw": dw}
    return {"dx" if kind == "dispatch_grad" else "out": y}
