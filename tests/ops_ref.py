"""64-bit definitions of the operators without an engine, on the device of their inputs, with the error each output may have.

Bounds.  A product of two 16-bit values is exact in fp32.  An fp32 sum of n terms, in any order and with one
rounding (or truncation) of at most 2^-23 per step, is off by at most (n + 8) 2^-23 times the sum of their
magnitudes.  exp, erfc and the divisions around them are off by a few units in the last place: 2^-19 of
the magnitudes they are multiplied with covers them.  The last rounding is half a step, eps/2 of the value
(and 2^-25 absolute where fp16 is subnormal)."""
import math

import torch

ACTS = ("none", "silu", "gelu", "gelu_tanh", "swiglu")
NONE, SILU, GELU, GELU_TANH, SWIGLU = range(5)
STEP = 2.0 ** -23
FUNC = 2.0 ** -19


def half_ulp(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    return 2.0 ** -25 if t == torch.float16 else 1e-38


def act64(z, act):
    if act == SILU:
        return z / (1 + torch.exp(-z))
    if act == GELU:
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if act == GELU_TANH:
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == SWIGLU:
        n = z.shape[1] // 2
        return act64(z[:, :n], SILU) * z[:, n:]
    return z


def dact64(z, act):
    if act == SILU:
        s = 1 / (1 + torch.exp(-z))
        return s + z * s * (1 - s)
    if act == GELU:
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == GELU_TANH:
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def dz64(dy, z, act):
    """dy * act'(z), and the magnitudes that an error of act' is multiplied with."""
    if act == SWIGLU:
        n = z.shape[1] // 2
        g, u = z[:, :n], z[:, n:]
        return (torch.cat([dy * u * dact64(g, SILU), dy * act64(g, SILU)], 1),
                torch.cat([dy.abs() * u.abs() * (1 + g.abs()), dy.abs() * (1 + g.abs())], 1))
    return dy * dact64(z, act), dy.abs() * (1 + z.abs())


def groups_of(offsets, m):
    """(group, rows) of a dense product (offsets None) or of every group."""
    if offsets is None:
        return [(None, slice(0, m))]
    off = offsets.tolist()
    return [(e, slice(off[e], off[e + 1])) for e in range(len(off) - 1)]


def matmul64(x, w, bias, act, residual, offsets, n):
    """(y, bound of its fp32 error, z, bound) in float64; rows in no group are zero."""
    m, k = x.shape
    nw = w.shape[-2]
    x, w = x.double(), w.double()
    z, ze = (torch.zeros(m, nw, dtype=torch.float64, device=x.device) for _ in range(2))
    for e, rows in groups_of(offsets, m):
        we = w if e is None else w[e]
        z[rows] = x[rows] @ we.t()
        mag = x[rows].abs() @ we.abs().t()
        if bias is not None:
            b = (bias if e is None else bias[e]).double()
            z[rows] += b
            mag = mag + b.abs()
        ze[rows] = (k + 8) * STEP * mag
    y = act64(z, act)
    if act == SWIGLU:
        g, u, ge, ue = z[:, :n], z[:, n:], ze[:, :n], ze[:, n:]
        ye = 1.1 * ge * (u.abs() + ue) + act64(g, SILU).abs() * ue + FUNC * (y.abs())
    else:
        ye = 1.2 * ze + (FUNC * y.abs() if act != NONE else 0)
    if residual is not None:
        r = residual.double()
        y = y + r
        ye = ye + STEP * (y.abs() + r.abs())
    return y, ye, z, ze


def assert_within(got, ref, err, what):
    """got (any type) against ref with err, plus the rounding of got's own type."""
    t = got.dtype
    g, ref, err = got.detach().cpu().double(), ref.cpu(), err.cpu()
    assert g.shape == ref.shape, what
    lim = (err + half_ulp(t) * (ref.abs() + err) + tiny(t)) if t != torch.float32 else err + STEP * ref.abs() + 1e-38
    off = (g - ref).abs()
    bad = ~(off <= lim)
    assert not bad.any(), "%s: %d of %d outside, worst %.3e where %.3e is allowed (value %.3e)" % (
        what, int(bad.sum()), bad.numel(), float(off[bad].max()), float(lim[bad][off[bad].argmax()]), float(ref[bad][off[bad].argmax()]))


def sort_ref(ids, E):
    """offsets, order, pos by the definition, one pair after the other."""
    flat = ids.reshape(-1).tolist()
    buckets = [[] for _ in range(E)]
    for p, e in enumerate(flat):
        if 0 <= e < E:
            buckets[e].append(p)
    offsets, order = [0], []
    for b in buckets:
        order += b
        offsets.append(len(order))
    pos = [-1] * len(flat)
    for place, p in enumerate(order):
        pos[p] = place
    order += [-1] * (len(flat) - len(order))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return i32(offsets), i32(order), i32(pos).view(ids.shape)
