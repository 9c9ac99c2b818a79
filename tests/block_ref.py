"""64-bit definitions of layer norm, the router's losses and microscaled 4-bit rows, with the error each output may have.

Bounds.  U = 2^-24 is half a step of fp32.  A sum whose terms pass through at most D additions is off by at most D U (1 + D U)
times the sum of their magnitudes, rounded up here to (D + 4) U.  A thread of a row adds at most max(64, H / 1024) values,
then come 6 steps over the wave and 16 over the waves: D below."""
import math

import torch

U = 2.0 ** -24
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def depth(H):
    return max(64, -(-H // 1024)) + 22


def norm64(x, w, b, eps):
    """(y, bound, mean, bound, rstd, bound)."""
    x = x.double()
    H, D = x.shape[1], depth(x.shape[1])
    mean = x.mean(1, keepdim=True)
    d = x - mean
    var = (d * d).mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    w = torch.ones(H, dtype=torch.float64) if w is None else w.double().to(x.device)
    b = torch.zeros(H, dtype=torch.float64) if b is None else b.double().to(x.device)
    y = d * rstd * w.to(x.device) + b.to(x.device)
    # deviations are taken from a first mean and their own mean put right: what is left of the mean is D U of mean |d|, d's own
    # rounding U |d|; the first mean is off by less than (D + 4) U mean |x|, which the deviations carry besides
    first = (D + 4) * U * x.abs().mean(1, keepdim=True)
    dabs = d.abs().mean(1, keepdim=True) + first
    em = (D + 6) * U * dabs
    # variance: relative (D + 8) U, and U of d in every square; 1 / sqrt: half of it and 4 U of its own
    rel = ((D + 10) * U * (var + first * first) + 2 * em * dabs) / (var + eps) + 4 * U
    ye = (w.abs().to(x.device) * rstd * ((d.abs() + first) * (rel + 6 * U) + em)) + 4 * U * (y.abs() + b.abs().to(x.device))
    return y, ye, mean, em + 2 * U * (mean.abs() + first), rstd, rstd * rel


def norm_grad64(dy, x, w, mean, rstd, residual):
    """(dx, bound, dw, bound, db, bound) for the statistics given."""
    dy, x = dy.double(), x.double()
    T, H = x.shape
    D, rows = depth(H), -(-T // 256) + 64
    mean, rstd = mean.double()[:, None], rstd.double()[:, None]
    xh = (x - mean) * rstd
    g = dy if w is None else dy * w.double()
    m1, m2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    a1, a2 = g.abs().mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
    dx = rstd * (g - m1 - xh * m2)
    err = rstd * (4 * U * g.abs() + (D + 8) * U * a1 + (D + 12) * U * xh.abs() * a2)
    if residual is not None:
        dx = dx + residual.double()
        err = err + U * (residual.double().abs() + dx.abs())
    return dx, err, (dy * xh).sum(0), (rows + 8) * U * (dy * xh).abs().sum(0), dy.sum(0), (rows + 4) * U * dy.abs().sum(0)


def balance64(logits, ids, mask, E):
    """(losses, bounds, counts, lse, bound)."""
    T, K = ids.shape
    x = logits.double()
    live = torch.ones(T, dtype=torch.bool) if mask is None else mask.clone()
    live &= ~(x == -math.inf).all(1)
    counts = torch.zeros(E + 1, dtype=torch.int64)
    for t in range(T):
        if live[t]:
            for i in ids[t].tolist():
                if 0 <= i < E:
                    counts[i] += 1
    counts[E] = n = int(live.sum())
    lse, le = torch.full((T,), -math.inf, dtype=torch.float64), torch.zeros(T, dtype=torch.float64)
    losses, errs = torch.zeros(2, dtype=torch.float64), torch.zeros(2, dtype=torch.float64)
    if n == 0:
        return losses, errs, counts, lse, le
    xl = x[live]
    lse[live] = torch.logsumexp(xl, 1)
    p = torch.softmax(xl, 1)
    top = xl.amax(1, keepdim=True)
    far = torch.where(xl == -math.inf, 0.0, top - xl)
    # exp: its argument is rounded (U |x - top|), itself good to 2 steps; sums of at most 64 + 6 steps; log to 2 steps
    pe = (far + 90) * U * p
    le[live] = pe.sum(1) + 4 * U * (1 + top[:, 0].abs() + lse[live].abs())
    f = counts[:E].double() / (n * K)
    rows = T // 1024 + 16
    losses[0] = E * (f * p.mean(0)).sum()
    errs[0] = E * (f * (pe.mean(0) + 90 * U * p.mean(0) + rows * U * p.mean(0))).sum() + 2 * U * losses[0]
    losses[1] = (lse[live] ** 2).mean()
    errs[1] = (2 * lse[live].abs() * le[live] + le[live] ** 2).mean() + (rows + 4) * U * losses[1]
    return losses, errs, counts, lse, le


def balance_grad64(logits, ids, counts, lse, dlosses, w, dw):
    """(dlogits, bound) from its parts, for the counts and lse given."""
    T, E = logits.shape
    K = ids.shape[1]
    x, lse = logits.double(), lse.double()
    live = lse > -math.inf
    out, err = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    n = int(counts[E])
    if dlosses is not None and n > 0:
        x = torch.where(live[:, None], x, 0.0)
        p = torch.where(live[:, None], torch.softmax(x, 1), 0.0)
        far = torch.where(x == -math.inf, 0.0, x.amax(1, keepdim=True) - x)
        f = counts[:E].double() / (n * K)
        s = (p * f).sum(1, keepdim=True)
        a, b = float(dlosses[0]) * E / n, 2 * float(dlosses[1]) / n
        z = torch.where(live, lse, 0.0)[:, None]
        out = p * (a * (f - s) + b * z)
        err = out.abs() * (far + 98) * U + p * (abs(a) * ((f + s) * 8 * U + (p * f * (far + 180)).sum(1, keepdim=True) * U) + 8 * U * (b * z).abs())
    if w is not None:
        w, dw = w.double(), dw.double()
        for t in range(T):
            ks = [k for k in range(K) if live[t] and 0 <= int(ids[t, k]) < E]
            s = sum(float(w[t, k] * dw[t, k]) for k in ks)
            mag = sum(abs(float(w[t, k] * dw[t, k])) for k in ks)
            for k in ks:
                out[t, ids[t, k]] += w[t, k] * (dw[t, k] - s)
                err[t, ids[t, k]] += (2 * K + 10) * U * abs(w[t, k]) * (abs(dw[t, k]) + mag)
    return out, err + 2 * U * out.abs()


# ---- 4-bit rows


def quantise(x):
    """Codes (a number each, [m, units * 128]) and scale bytes of x [m,k], value by value from the definition."""
    m, k = x.shape
    units = -(-k // 128)
    pad = torch.zeros(m, units * 128, dtype=torch.float64)
    pad[:, :k] = x.double()
    b = pad.view(m, -1, 32)
    top = b.abs().amax(2)
    bad = ~torch.isfinite(b).all(2)
    mant, e = torch.frexp(torch.where(bad | (top == 0), torch.ones_like(top), top))   # top = mant 2^e, mant in [0.5, 1)
    e = torch.where(top == 0, -127, torch.clamp(e.to(torch.int64) - 3, -127, 127))
    v = torch.where(bad[..., None], torch.zeros_like(b), torch.ldexp(b, -e[..., None].double()))
    table = torch.tensor(E2M1, dtype=torch.float64)
    off = (v.abs()[..., None] - table).abs()
    best = off.amin(3, keepdim=True)
    near = off == best
    # of two that are as near the even code
    code = torch.where(near.sum(3) > 1, (near & (torch.arange(8) % 2 == 0)).to(torch.uint8).argmax(3), near.to(torch.uint8).argmax(3))
    sign = torch.signbit(v) & ~bad[..., None]
    return (code + 8 * sign).view(m, -1), torch.where(bad, 255, e + 127).to(torch.uint8)


def pack(codes):
    codes = codes.to(torch.uint8)
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def values(q, scales):
    """float64 values of packed codes [.., units * 64] and scales [.., units * 4]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=q.device)
    c = torch.stack([q & 15, q >> 4], -1).view(*q.shape[:-1], 2 * q.shape[-1]).long()
    s = torch.where(scales == 255, math.nan, torch.ldexp(torch.ones_like(scales, dtype=torch.float64), scales.double() - 127))
    return table[c] * s.repeat_interleave(32, -1)
