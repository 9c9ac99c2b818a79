"""Operators around the routed-expert step that need no engine: dense products with their epilogue, the
experts' products on sorted rows, tokens sorted by expert and back, and the gradients of all of them.

Every call enqueues on `stream` (a torch.cuda.Stream, a handle, or None for the current stream of the
tensors' device), writes the outputs it is given and keeps nothing.  Matrices need unit stride inside a row;
any stride between rows works for inputs (0 broadcasts a row) and any that keeps rows apart for outputs.
A wrong type, shape, stride or device raises EffError (EFF_EINVAL) before anything is launched.

torch's autograd records none of these calls, whether inputs require grad or not: a training step calls the *_backward
functions itself.  Outputs count as written in place (their versions go up), so a graph that saved one refuses its
backward pass, as after a torch operation with out=.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import ACT_NONE, ACT_SWIGLU, EFF_EINVAL, EffError, lib

_DT = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_HALF = {torch.bfloat16: 0, torch.float16: 1}
_I32, _F32 = torch.int32, torch.float32
_MAX_GROUPS, _MAX_TOPK = 4096, 32         # the library's own bounds; its counts are 32-bit
_written = torch._C._increment_version    # takes tensors in a tuple or list; those of inference mode have no version


class MatmulDesc(ctypes.Structure):
    """eff_matmul_desc"""
    _fields_ = [("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("act", ctypes.c_int32),
                ("groups", ctypes.c_int32)] + [(n, ctypes.c_int64) for n in (
                    "m", "n", "k", "ld_x", "ld_w", "ld_y", "ld_residual", "ld_pre", "stride_w", "ld_dx", "ld_dw",
                    "stride_dw")]


_pack_desc = struct.Struct("=4i12q").pack   # the same bytes, packed faster than a ctypes structure is filled


def _bad(msg: str):
    raise EffError(EFF_EINVAL, msg)


# The checks below run in front of calls of a few microseconds: few attribute accesses, no torch objects made, and
# something that is no tensor shows as the AttributeError that _no_tensor turns into an EffError.

def _no_tensor(e: AttributeError):
    raise EffError(EFF_EINVAL, "an argument is not a tensor (%s)" % e) from e


def _matrix(name, t, dtype, rows, cols, dev, out=False):
    """Checks a row-major matrix; returns its address and the elements between rows."""
    if t.dtype is not dtype or t.shape != (rows, cols):
        _explain(name, t, dtype, (rows, cols))
    if t.get_device() != dev:
        _bad("%s is on %s, the call on GPU %d" % (name, t.device, dev))
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        _bad("%s must have unit stride inside a row" % name)
    if rows <= 1:
        ld = cols
    elif out and ld < cols:
        _bad("rows of %s overlap" % name)
    return t.data_ptr(), ld


def _stack(name, t, dtype, groups, rows, cols, dev, out=False):
    """A matrix per group: its address, the elements between rows and between groups."""
    if t.dtype is not dtype or t.shape != (groups, rows, cols):
        _explain(name, t, dtype, (groups, rows, cols))
    if t.get_device() != dev:
        _bad("%s is on %s, the call on GPU %d" % (name, t.device, dev))
    between, ld, unit = t.stride()
    if unit != 1 and cols > 1:
        _bad("%s must have unit stride inside a row" % name)
    if rows <= 1:
        ld = cols
    if groups <= 1:
        between = ld * rows
    if out and (ld < cols or between < ld * (rows - 1) + cols):
        _bad("rows of %s overlap" % name)
    return t.data_ptr(), ld, between


def _dense(name, t, dtype, shape, dev):
    if t.dtype is not dtype or t.shape != shape:
        _explain(name, t, dtype, shape)
    if t.get_device() != dev:
        _bad("%s is on %s, the call on GPU %d" % (name, t.device, dev))
    if not t.is_contiguous():
        _bad("%s must be contiguous" % name)
    return t.data_ptr()


def _explain(name, t, dtype, shape):
    if not isinstance(t, torch.Tensor):
        _bad("%s must be a tensor" % name)
    _bad("%s must be %s of shape %s, got %s of %s" % (name, dtype, tuple(shape), t.dtype, tuple(t.shape)))


def _device(name, t):
    """The GPU the call runs on."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _bad("%s must be a tensor on the GPU" % name)
    return t.get_device()


def _call(fn, dev, stream, args, need=None):
    """Runs fn(*args[, workspace, bytes], stream) with the tensors' device current; need: workspace bytes, or None for
    a call without one."""
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return _call(fn, dev, stream, args, need)
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(dev)
    elif isinstance(stream, int):
        handle = stream
    else:
        handle = stream.cuda_stream
        if stream.device_index != dev:
            _bad("the stream is on GPU %d, the tensors on GPU %d" % (stream.device_index, dev))
    if need is None:
        rc = fn(*args, handle)
    elif need <= 0:      # a negative number is the description's error: the call itself reports it
        rc = fn(*args, None, 0, handle)
    elif stream is None:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        rc = fn(*args, ws.data_ptr(), need, handle)
    else:                # memory that the caching allocator orders with that stream
        with torch.cuda.stream(torch.cuda.ExternalStream(handle, device=dev) if isinstance(stream, int) else stream):
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
        rc = fn(*args, ws.data_ptr(), need, handle)
    if rc != 0:
        raise EffError(rc, lib().eff_last_error().decode())


def _sizes(x, w, act, grouped):
    """(m, n, k, rows of one W, groups) of a product, from x [m,k] and w ([nw,k] or [E,nw,k])."""
    if x.dtype not in _HALF:
        _bad("x must be bfloat16 or float16, got %s" % x.dtype)
    xs, ws = x.shape, w.shape
    if len(xs) != 2 or len(ws) != (3 if grouped else 2):
        _bad("x must be [m,k] and w %s" % ("[E,n,k]" if grouped else "[n,k]"))
    nw, groups = ws[-2], ws[0] if grouped else 0
    if act == ACT_NONE or act in (1, 2, 3):
        return xs[0], nw, xs[1], nw, groups
    if act != ACT_SWIGLU:
        _bad("unknown activation %r" % (act,))
    if nw % 2:
        _bad("w needs an even number of rows (gate, then up) with ACT_SWIGLU")
    return xs[0], nw // 2, xs[1], nw, groups


def _weights(w, dt, groups, nw, k, dev, offsets):
    if offsets is None:
        return _matrix("w", w, dt, nw, k, dev) + (0, None)
    if not 1 <= groups <= _MAX_GROUPS:
        _bad("w needs 1 to %d groups" % _MAX_GROUPS)
    return _stack("w", w, dt, groups, nw, k, dev) + (_dense("offsets", offsets, _I32, (groups + 1,), dev),)


def _out_type(name, t, dt):
    got = t.dtype
    if got is not dt and got is not _F32:
        _bad("%s must be a tensor of x's type or float32" % name)
    return got


def _forward(x, w, offsets, y, bias, act, residual, pre, stream):
    try:
        dev = _device("x", x)
        dt = x.dtype
        m, n, k, nw, groups = _sizes(x, w, act, offsets is not None)
        yt = _out_type("y", y, dt)
        px, ldx = _matrix("x", x, dt, m, k, dev)
        pw, ldw, sw, po = _weights(w, dt, groups, nw, k, dev, offsets)
        py, ldy = _matrix("y", y, yt, m, n, dev, True)
        pb = pr = pp = None
        ldr, ldp = 0, nw
        if bias is not None:
            pb = _dense("bias", bias, dt, (nw,) if offsets is None else (groups, nw), dev)
        if residual is not None:
            pr, ldr = _matrix("residual", residual, dt, m, n, dev)
        if pre is not None:
            pp, ldp = _matrix("pre", pre, dt, m, nw, dev, True)
        d = _pack_desc(_HALF[dt], _DT[yt], act, groups, m, n, k, ldx, ldw, ldy, ldr, ldp, sw, 0, 0, 0)
        L = lib()
        _call(L.eff_matmul, dev, stream, (d, px, pw, pb, pr, po, py, pp), L.eff_matmul_workspace(d, 0))
        _written((y,) if pre is None else (y, pre))
    except AttributeError as e:
        _no_tensor(e)
    except struct.error as e:
        _bad("act or a size is not an integer that the description holds (%s)" % e)


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
    try:
        dev = _device("x", x)
        dt = x.dtype
        m, n, k, nw, groups = _sizes(x, w, act, offsets is not None)
        dyt = _out_type("dy", dy, dt)
        px, ldx = _matrix("x", x, dt, m, k, dev)
        pw, ldw, sw, po = _weights(w, dt, groups, nw, k, dev, offsets)
        pdy, lddy = _matrix("dy", dy, dyt, m, n, dev)
        pp = pdx = pdw = pdb = None
        ldp, lddx, lddw, sdw = nw, k, k, 0
        if pre is not None:
            pp, ldp = _matrix("pre", pre, dt, m, nw, dev)
        elif act != ACT_NONE:
            _bad("pre is needed with an activation")
        if dx is not None:
            pdx, lddx = _matrix("dx", dx, dt, m, k, dev, True)
        if dw is not None:
            if offsets is None:
                pdw, lddw = _matrix("dw", dw, dt, nw, k, dev, True)
            else:
                pdw, lddw, sdw = _stack("dw", dw, dt, groups, nw, k, dev, True)
        if dbias is not None:
            pdb = _dense("dbias", dbias, dt, (nw,) if offsets is None else (groups, nw), dev)
        d = _pack_desc(_HALF[dt], _DT[dyt], act, groups, m, n, k, ldx, ldw, lddy, 0, ldp, sw, lddx, lddw, sdw)
        L = lib()
        _call(L.eff_matmul_backward, dev, stream, (d, pdy, px, pw, pp, po, pdx, pdw, pdb), L.eff_matmul_workspace(d, 1))
        _written([t for t in (dx, dw, dbias) if t is not None])
    except AttributeError as e:
        _no_tensor(e)
    except struct.error as e:
        _bad("act or a size is not an integer that the description holds (%s)" % e)


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
    try:
        dev = _device("ids", ids)
        if offsets.dim() != 1 or not 2 <= offsets.shape[0] <= _MAX_GROUPS + 1:
            _bad("offsets must be a vector of E+1 values, E from 1 to %d" % _MAX_GROUPS)
        n, E, shape = ids.numel(), offsets.shape[0] - 1, ids.shape
        pi = _dense("ids", ids, _I32, shape, dev)
        po = _dense("offsets", offsets, _I32, (E + 1,), dev)
        pr = _dense("order", order, _I32, (n,), dev)
        pp = _dense("pos", pos, _I32, shape, dev)
        L = lib()
        _call(L.eff_sort_tokens, dev, stream, (pi, n, E, po, pr, pp), L.eff_sort_tokens_workspace(n, E))
        _written((offsets, order, pos))
    except AttributeError as e:
        _no_tensor(e)


def _rows_of(name, t):
    """(rows, H) of a matrix of token or expert rows."""
    shape = t.shape
    if len(shape) != 2 or t.dtype not in _DT:
        _bad("%s must be a matrix of bfloat16, float16 or float32" % name)
    return shape


def _pos(pos, T, dev):
    shape = pos.shape
    if len(shape) != 2 or shape[0] != T:
        _bad("pos must be [T,K] with T = %d" % T)
    if shape[1] > _MAX_TOPK:
        _bad("pos has more than %d places a token" % _MAX_TOPK)
    return _dense("pos", pos, _I32, shape, dev), shape[1]


def dispatch_tokens(x, pos, xs, stream=None):
    """eff_dispatch_tokens: xs[pos[t,k]] = x[t] for every routed pair; the other rows of xs stay as they were.
    x [T,H], xs [rows,H] (bfloat16, float16 or float32), pos int32 [T,K] from sort_tokens."""
    try:
        dev = _device("x", x)
        T, H = _rows_of("x", x)
        R = _rows_of("xs", xs)[0]
        px, ldx = _matrix("x", x, x.dtype, T, H, dev)
        ps, lds = _matrix("xs", xs, x.dtype, R, H, dev, True)
        pp, K = _pos(pos, T, dev)
        _call(lib().eff_dispatch_tokens, dev, stream, (_DT[x.dtype], px, ldx, pp, T, K, H, ps, lds, R))
        _written((xs,))
    except AttributeError as e:
        _no_tensor(e)


def dispatch_tokens_backward(dxs, pos, dx, stream=None):
    """eff_dispatch_tokens_backward: dx[t] = sum over k of dxs[pos[t,k]] over the routed pairs."""
    try:
        dev = _device("dxs", dxs)
        R, H = _rows_of("dxs", dxs)
        T = _rows_of("dx", dx)[0]
        ps, lds = _matrix("dxs", dxs, dxs.dtype, R, H, dev)
        px, ldx = _matrix("dx", dx, dxs.dtype, T, H, dev, True)
        pp, K = _pos(pos, T, dev)
        _call(lib().eff_dispatch_tokens_backward, dev, stream, (_DT[dxs.dtype], ps, lds, R, pp, T, K, H, px, ldx))
        _written((dx,))
    except AttributeError as e:
        _no_tensor(e)


def combine_tokens(ys, pos, w, out, residual=None, stream=None):
    """eff_combine_tokens: out[t] = residual[t] + sum over k of w[t,k] * ys[pos[t,k]] over the routed pairs.
    ys [rows,H], out and residual [T,H] of one type, w float32 [T,K].  out may be residual."""
    try:
        dev = _device("ys", ys)
        R, H = _rows_of("ys", ys)
        T = _rows_of("out", out)[0]
        py, ldy = _matrix("ys", ys, ys.dtype, R, H, dev)
        po, ldo = _matrix("out", out, ys.dtype, T, H, dev, True)
        pr, ldr = _matrix("residual", residual, ys.dtype, T, H, dev) if residual is not None else (None, 0)
        pp, K = _pos(pos, T, dev)
        pw = _dense("w", w, _F32, (T, K), dev)
        _call(lib().eff_combine_tokens, dev, stream, (_DT[ys.dtype], py, ldy, R, pp, pw, T, K, H, pr, ldr, po, ldo))
        _written((out,))
    except AttributeError as e:
        _no_tensor(e)


def combine_tokens_backward(dout, ys, pos, w, dys, dw=None, stream=None):
    """eff_combine_tokens_backward: dys[pos[t,k]] = w[t,k] * dout[t] (the other rows of dys stay as they were) and, if
    given, dw[t,k] = <dout[t], ys[pos[t,k]]> in float32 (0 for an unrouted pair).  The residual's gradient is dout."""
    try:
        dev = _device("dout", dout)
        T, H = _rows_of("dout", dout)
        R = _rows_of("ys", ys)[0]
        pd, ldd = _matrix("dout", dout, dout.dtype, T, H, dev)
        py, ldy = _matrix("ys", ys, dout.dtype, R, H, dev)
        ps, lds = _matrix("dys", dys, dout.dtype, R, H, dev, True)
        pp, K = _pos(pos, T, dev)
        pw = _dense("w", w, _F32, (T, K), dev)
        pg = _dense("dw", dw, _F32, (T, K), dev) if dw is not None else None
        _call(lib().eff_combine_tokens_backward, dev, stream,
              (_DT[dout.dtype], pd, ldd, py, ldy, R, pp, pw, T, K, H, ps, lds, pg))
        _written((dys,) if dw is None else (dys, dw))
    except AttributeError as e:
        _no_tensor(e)