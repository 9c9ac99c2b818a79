"""Operators around the routed-expert step that need no engine: dense products with their epilogue, the
experts' products on sorted rows, tokens sorted by expert and back, and the gradients of all of them.

Every call enqueues on `stream` (a torch.cuda.Stream, a handle, or None for the current stream of the
tensors' device), writes the outputs it is given and keeps nothing.  Matrices need unit stride inside a row;
any stride between rows works for inputs (0 broadcasts a row) and any that keeps rows apart for outputs.
A wrong type, shape, stride or device raises EffError (EFF_EINVAL) before anything is launched.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import ACT_NONE, ACT_SWIGLU, EFF_EINVAL, EffError, lib

_DT = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_HALF = (torch.bfloat16, torch.float16)


class MatmulDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("act", ctypes.c_int32),
                ("groups", ctypes.c_int32)] + [(n, ctypes.c_int64) for n in (
                    "m", "n", "k", "ld_x", "ld_w", "ld_y", "ld_residual", "ld_pre", "stride_w", "ld_dx", "ld_dw",
                    "stride_dw")]


def _bad(msg: str):
    raise EffError(EFF_EINVAL, msg)


def _tensor(name, t, dtype, shape, device):
    """Checks one tensor; returns its address."""
    if not isinstance(t, torch.Tensor):
        _bad("%s must be a tensor" % name)
    if t.dtype != dtype:
        _bad("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        _bad("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.device != device:
        _bad("%s is on %s, the call on %s" % (name, t.device, device))
    return t.data_ptr()


def _matrix(name, t, dtype, shape, device, out=False):
    """Checks a row-major matrix (or stack of them); returns its address and the elements between rows."""
    p = _tensor(name, t, dtype, shape, device)
    rows, cols = shape[-2], shape[-1]
    st = t.stride()
    if cols > 1 and st[-1] != 1:
        _bad("%s must have unit stride inside a row" % name)
    ld = st[-2] if rows > 1 else cols
    if out and ld < cols:
        _bad("rows of %s overlap" % name)
    return p, ld


def _dense(name, t, dtype, shape, device):
    p = _tensor(name, t, dtype, shape, device)
    if not t.is_contiguous():
        _bad("%s must be contiguous" % name)
    return p


def _device(name, t):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _bad("%s must be a tensor on the GPU" % name)
    return t.device


@contextlib.contextmanager
def _on(device, stream):
    with torch.cuda.device(device):
        yield torch.cuda.current_stream().cuda_stream if stream is None else \
            stream if isinstance(stream, int) else stream.cuda_stream


def _stream(device, stream):
    """The stream's handle where `device` is the current one, else None (the call then runs under _on)."""
    if device.index != torch.cuda.current_device():
        return None
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _workspace(nbytes, device, stream, handle):
    """nbytes of device memory that the caching allocator orders with `stream`."""
    if nbytes <= 0:
        return None
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    s = stream if not isinstance(stream, int) else torch.cuda.ExternalStream(handle, device=device)
    with torch.cuda.stream(s):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _call(fn, device, stream, args, need=0):
    """Runs fn(*args[, workspace, bytes], stream) with the tensors' device current."""
    handle = _stream(device, stream)
    if handle is None:
        with _on(device, stream) as handle:
            return _run(fn, device, stream, handle, args, need)
    return _run(fn, device, stream, handle, args, need)


def _run(fn, device, stream, handle, args, need):
    if need is None:
        rc = fn(*args, handle)
    else:
        ws = _workspace(need, device, stream, handle)
        rc = fn(*args, None if ws is None else ws.data_ptr(), max(0, need), handle)
    if rc != 0:
        raise EffError(rc, lib().eff_last_error().decode())


def _sizes(x, w, act, grouped):
    """(m, n, k, rows of one W, groups) of a product, from x [m,k] and w ([nw,k] or [E,nw,k])."""
    if x.dtype not in _HALF:
        _bad("x must be bfloat16 or float16, got %s" % x.dtype)
    if x.dim() != 2 or not isinstance(w, torch.Tensor) or w.dim() != (3 if grouped else 2):
        _bad("x must be [m,k] and w %s" % ("[E,n,k]" if grouped else "[n,k]"))
    nw = w.shape[-2]
    if act not in (0, 1, 2, 3, 4):
        _bad("unknown activation %r" % (act,))
    if act == ACT_SWIGLU and nw % 2:
        _bad("w needs an even number of rows (gate, then up) with ACT_SWIGLU")
    return x.shape[0], nw // 2 if act == ACT_SWIGLU else nw, x.shape[1], nw, w.shape[0] if grouped else 0


def _offsets(offsets, groups, dev):
    return _dense("offsets", offsets, torch.int32, (groups + 1,), dev) if groups else None


def _forward(x, w, offsets, y, bias, act, residual, pre, stream):
    dev = _device("x", x)
    m, n, k, nw, groups = _sizes(x, w, act, offsets is not None)
    dt = x.dtype
    lead = (groups,) if offsets is not None else ()
    px, ldx = _matrix("x", x, dt, (m, k), dev)
    pw, ldw = _matrix("w", w, dt, lead + (nw, k), dev)
    if not isinstance(y, torch.Tensor) or y.dtype not in (dt, torch.float32):
        _bad("y must be a tensor of x's type or float32")
    py, ldy = _matrix("y", y, y.dtype, (m, n), dev, out=True)
    pb = _dense("bias", bias, dt, lead + (nw,), dev) if bias is not None else None
    pr, ldr = _matrix("residual", residual, dt, (m, n), dev) if residual is not None else (None, 0)
    pp, ldp = _matrix("pre", pre, dt, (m, nw), dev, out=True) if pre is not None else (None, nw)
    d = MatmulDesc(_DT[dt], _DT[y.dtype], act, groups, m, n, k, ldx, ldw, ldy, ldr, ldp, w.stride(0) if lead else 0, 0, 0, 0)
    L, pd = lib(), ctypes.addressof(d)
    _call(L.eff_matmul, dev, stream, (pd, px, pw, pb, pr, _offsets(offsets, groups, dev), py, pp), L.eff_matmul_workspace(pd, 0))


def matmul(x, w, y, bias=None, act=ACT_NONE, residual=None, pre=None, stream=None):
    """eff_matmul: y = act(x @ w.T + bias) + residual.  x [m,k], w [n,k] ([2n,k] with ACT_SWIGLU, gate rows then up
    rows), bias [rows of w], residual [m,n], all bfloat16 or all float16; y [m,n] of that type or float32, written;
    pre [m, rows of w], written if given: the sums before the activation, for matmul_backward.  y may be residual."""
    _forward(x, w, None, y, bias, act, residual, pre, stream)


def grouped_matmul(x, w, offsets, y, bias=None, act=ACT_NONE, residual=None, pre=None, stream=None):
    """eff_matmul with groups: rows offsets[e]..offsets[e+1]-1 of x [m,k] with w[e], w [E,n,k] (bias [E,n]); offsets
    int32 [E+1] as sort_tokens writes them.  Rows in no group are not read and their rows of y and pre stay as they were."""
    if offsets is None:
        _bad("offsets are needed")
    _forward(x, w, offsets, y, bias, act, residual, pre, stream)


def _backward(dy, x, w, offsets, dx, dw, dbias, act, pre, stream):
    dev = _device("x", x)
    m, n, k, nw, groups = _sizes(x, w, act, offsets is not None)
    dt = x.dtype
    lead = (groups,) if offsets is not None else ()
    px, ldx = _matrix("x", x, dt, (m, k), dev)
    pw, ldw = _matrix("w", w, dt, lead + (nw, k), dev)
    if not isinstance(dy, torch.Tensor) or dy.dtype not in (dt, torch.float32):
        _bad("dy must be a tensor of x's type or float32")
    pdy, lddy = _matrix("dy", dy, dy.dtype, (m, n), dev)
    if act != ACT_NONE and pre is None:
        _bad("pre is needed with an activation")
    pp, ldp = _matrix("pre", pre, dt, (m, nw), dev) if pre is not None else (None, nw)
    pdx, lddx = _matrix("dx", dx, dt, (m, k), dev, out=True) if dx is not None else (None, k)
    pdw, lddw = _matrix("dw", dw, dt, lead + (nw, k), dev, out=True) if dw is not None else (None, k)
    pdb = _dense("dbias", dbias, dt, lead + (nw,), dev) if dbias is not None else None
    d = MatmulDesc(_DT[dt], _DT[dy.dtype], act, groups, m, n, k, ldx, ldw, lddy, 0, ldp, w.stride(0) if lead else 0, lddx,
                   lddw, dw.stride(0) if lead and dw is not None else 0)
    L, pd = lib(), ctypes.addressof(d)
    _call(L.eff_matmul_backward, dev, stream,
          (pd, pdy, px, pw, pp, _offsets(offsets, groups, dev), pdx, pdw, pdb), L.eff_matmul_workspace(pd, 1))


def matmul_backward(dy, x, w, dx=None, dw=None, dbias=None, act=ACT_NONE, pre=None, stream=None):
    """eff_matmul_backward: from dy [m,n] (x's type, or float32 if y was), the forward's x and w and, with an
    activation, its pre, writes the gradients that are given: dx [m,k], dw like w, dbias [rows of w].  The
    residual's gradient is dy itself."""
    _backward(dy, x, w, None, dx, dw, dbias, act, pre, stream)


def grouped_matmul_backward(dy, x, w, offsets, dx=None, dw=None, dbias=None, act=ACT_NONE, pre=None, stream=None):
    """The gradients of grouped_matmul.  A group without rows gets zeros in dw and dbias; rows of dx in no group stay as
    they were."""
    if offsets is None:
        _bad("offsets are needed")
    _backward(dy, x, w, offsets, dx, dw, dbias, act, pre, stream)


def sort_tokens(ids, offsets, order, pos, stream=None):
    """eff_sort_tokens: ids int32 (any shape, contiguous; [T,K] as route writes them) sorted stably by expert.  Writes
    offsets int32 [E+1] (its length says E), order int32 [pairs] (pair at a place, -1 behind the last) and pos int32,
    shaped like ids (place of a pair, -1 for an id outside [0,E))."""
    dev = _device("ids", ids)
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 2:
        _bad("offsets must be a vector of E+1 values")
    n, E = ids.numel(), offsets.shape[0] - 1
    pi = _dense("ids", ids, torch.int32, ids.shape, dev)
    po = _dense("offsets", offsets, torch.int32, (E + 1,), dev)
    pr = _dense("order", order, torch.int32, (n,), dev)
    pp = _dense("pos", pos, torch.int32, ids.shape, dev)
    L = lib()
    need = L.eff_sort_tokens_workspace(n, E)
    _call(L.eff_sort_tokens, dev, stream, (pi, n, E, po, pr, pp), need)


def _rows_of(name, t, dev):
    """(rows, H) of a matrix of token or expert rows."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.dtype not in _DT:
        _bad("%s must be a matrix of bfloat16, float16 or float32" % name)
    return t.shape


def _pos(pos, T, dev):
    if not isinstance(pos, torch.Tensor) or pos.dim() != 2 or pos.shape[0] != T:
        _bad("pos must be [T,K] with T = %d" % T)
    return _dense("pos", pos, torch.int32, pos.shape, dev), pos.shape[1]


def dispatch_tokens(x, pos, xs, stream=None):
    """eff_dispatch_tokens: xs[pos[t,k]] = x[t] for every routed pair; the other rows of xs stay as they were.
    x [T,H], xs [rows,H] (bfloat16, float16 or float32), pos int32 [T,K] from sort_tokens."""
    dev = _device("x", x)
    T, H = _rows_of("x", x, dev)
    R = _rows_of("xs", xs, dev)[0]
    px, ldx = _matrix("x", x, x.dtype, (T, H), dev)
    ps, lds = _matrix("xs", xs, x.dtype, (R, H), dev, out=True)
    pp, K = _pos(pos, T, dev)
    _call(lib().eff_dispatch_tokens, dev, stream, (_DT[x.dtype], px, ldx, pp, T, K, H, ps, lds, R), None)


def dispatch_tokens_backward(dxs, pos, dx, stream=None):
    """eff_dispatch_tokens_backward: dx[t] = sum over k of dxs[pos[t,k]] over the routed pairs."""
    dev = _device("dxs", dxs)
    R, H = _rows_of("dxs", dxs, dev)
    T = _rows_of("dx", dx, dev)[0]
    ps, lds = _matrix("dxs", dxs, dxs.dtype, (R, H), dev)
    px, ldx = _matrix("dx", dx, dxs.dtype, (T, H), dev, out=True)
    pp, K = _pos(pos, T, dev)
    _call(lib().eff_dispatch_tokens_backward, dev, stream, (_DT[dxs.dtype], ps, lds, R, pp, T, K, H, px, ldx), None)


def combine_tokens(ys, pos, w, out, residual=None, stream=None):
    """eff_combine_tokens: out[t] = residual[t] + sum over k of w[t,k] * ys[pos[t,k]] over the routed pairs.
    ys [rows,H], out and residual [T,H] of one type, w float32 [T,K].  out may be residual."""
    dev = _device("ys", ys)
    R, H = _rows_of("ys", ys, dev)
    T = _rows_of("out", out, dev)[0]
    py, ldy = _matrix("ys", ys, ys.dtype, (R, H), dev)
    po, ldo = _matrix("out", out, ys.dtype, (T, H), dev, out=True)
    pr, ldr = _matrix("residual", residual, ys.dtype, (T, H), dev) if residual is not None else (None, 0)
    pp, K = _pos(pos, T, dev)
    pw = _dense("w", w, torch.float32, (T, K), dev)
    _call(lib().eff_combine_tokens, dev, stream, (_DT[ys.dtype], py, ldy, R, pp, pw, T, K, H, pr, ldr, po, ldo), None)


def combine_tokens_backward(dout, ys, pos, w, dys, dw=None, stream=None):
    """eff_combine_tokens_backward: dys[pos[t,k]] = w[t,k] * dout[t] (the other rows of dys stay as they were) and, if
    given, dw[t,k] = <dout[t], ys[pos[t,k]]> in float32 (0 for an unrouted pair).  The residual's gradient is dout."""
    dev = _device("dout", dout)
    T, H = _rows_of("dout", dout, dev)
    R = _rows_of("ys", ys, dev)[0]
    pd, ldd = _matrix("dout", dout, dout.dtype, (T, H), dev)
    py, ldy = _matrix("ys", ys, dout.dtype, (R, H), dev)
    ps, lds = _matrix("dys", dys, dout.dtype, (R, H), dev, out=True)
    pp, K = _pos(pos, T, dev)
    pw = _dense("w", w, torch.float32, (T, K), dev)
    pg = _dense("dw", dw, torch.float32, (T, K), dev) if dw is not None else None
    _call(lib().eff_combine_tokens_backward, dev, stream,
          (_DT[dout.dtype], pd, ldd, py, ldy, R, pp, pw, T, K, H, ps, lds, pg), None)
