"""Binding of what stands around a block in a stack: the residual's addition with its RMS norm, the
projections in 8 bits, and the clipping of a step's gradients (see include/m2rnn.h for the formulas).

Checks, allocation, streams and devices are as in the selective block's binding: outputs and workspaces
are torch memory, made when they are not given, and the calls run on the current CUDA stream unless the
keyword ``stream`` names another.

8-bit tensors are float8_e4m3fn with one float8_e8m0fnu scale (a power of two) for each 128 channels, for
weights for each 128 x 128.  Their rows start on 16-byte boundaries; what is made here is laid out so.
"""
from __future__ import annotations

from array import array

import torch

from .m2rnn import OK, load_library
from .ssm import BF16, F32, _device, _on_stream, _ptr, _raise, _refuse, _sizes, _stream, _workspace

FP8, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def _rows(t, name, dtype, shape, dev):
    """The address of a tensor [..., D] of this type and shape whose rows lie one stride apart, each
    contiguous, and that stride in elements."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _refuse(t, name, dtype, shape, dev)
    if t.is_contiguous():
        return t.data_ptr(), shape[-1]
    s = t.stride()
    if t.numel() == 0:
        return t.data_ptr(), shape[-1]
    if s[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"{name}: the channels of a row must be contiguous")
    row = count = None  # from row to row; rows so far
    for i in range(len(shape) - 2, -1, -1):
        if shape[i] == 1:
            continue
        if row is None:
            row, count = s[i], shape[i]
        elif s[i] == row * count:
            count *= shape[i]
        else:
            raise ValueError(f"{name}: rows must lie one stride apart")
    return t.data_ptr(), shape[-1] if row is None else row


def _byte_rows(t, name, shape, dev):
    """The same for e4m3 values, whose rows start on 16-byte boundaries."""
    p, row = _rows(t, name, FP8, shape, dev)
    if t.numel() <= shape[-1]:  # a single row, or none: nothing lies behind it
        row = (shape[-1] + 15) // 16 * 16
    if p % 16 or row % 16:
        raise ValueError(f"{name}: rows must start on 16-byte boundaries; {row} bytes apart from address {p:#x} they "
                         "do not (the package's own 8-bit tensors do)")
    return p, row


def _dense(like, dtype):
    """A new dense tensor of the same shape (the like-form of empty is the cheapest)."""
    if like.dtype is dtype and like.is_contiguous():
        return torch.empty_like(like)
    return torch.empty(like.shape, dtype=dtype, device=like.device)


def _new_bytes(like, shape):
    """An e4m3 tensor whose rows start on 16-byte boundaries, those of more than 128 values on 128-byte ones (the
    product reads 128 bytes of a row at a time, which then lie in one line of the cache), its address and the
    bytes from row to row."""
    D = shape[-1]
    to = 128 if D > 128 else 16
    row = (D + to - 1) // to * to
    if D == row:
        t = torch.empty(shape, dtype=FP8, device=like.device)
    else:
        strides = [1]
        for n in reversed(shape[1:]):
            strides.append(row if len(strides) == 1 else strides[-1] * n)
        t = torch.empty_strided(shape, strides[::-1], dtype=FP8, device=like.device)
    return t, t.data_ptr(), row


def _blocks(n):
    return (n + 127) // 128


# ---------------------------------------------------------------- residual RMS norm
# Tensors that are made here need no check: a token's call is short.
def _norm_args(x, residual, w, h):
    """Checks the norm's inputs: (device, h, sizes, arguments up to w, address of h)."""
    dev = _device(x)
    shape = x.shape
    D = shape[-1]
    _sizes(D)
    if residual is None:
        kind = x.dtype
        if kind is not BF16 and kind is not F32:
            raise TypeError(f"x: expected {F32} or {BF16}, got {kind}")
        if h is not None:
            raise ValueError("h: without a residual it is x")
        sp, row = _rows(x, "x", kind, shape, dev)
        args, h, hp = (None, 0, sp, kind is F32, row), x, None
    else:
        kind = residual.dtype
        if kind is not BF16 and kind is not F32:
            raise TypeError(f"residual: expected {F32} or {BF16}, got {kind}")
        xp, x_row = _rows(x, "x", BF16, shape, dev)
        sp, row = _rows(residual, "residual", kind, shape, dev)
        if h is None:
            h = _dense(residual, kind)
            hp = h.data_ptr()
        else:
            hp = _ptr(h, "h", kind, shape, dev)
        args = (xp, x_row, sp, kind is F32, row)
    return dev, h, (x.numel() // D if D else 0, D), (*args, _ptr(w, "w", F32, (D,), dev)), hp


@_on_stream
def add_rmsnorm(x, residual, w, eps=1e-5, out=None, h=None):
    """RMS norm of a residual stream: h = residual + x in the residual's type, out = h /
    sqrt(mean(h^2) + eps) times w.  x [..., D] bf16, residual [..., D] bf16 or float32 (rows of both may lie
    a wider stride apart), w [D] float32; residual None: h is x, bf16 or float32.  ``h`` may be the residual
    itself (in place).  Returns (out [..., D] bf16, h)."""
    dev, h, size, args, hp = _norm_args(x, residual, w, h)
    if out is None:
        out = _dense(x, BF16)
        op = out.data_ptr()
    else:
        op = _ptr(out, "out", BF16, x.shape, dev)
    st = load_library().m2rnn_add_rmsnorm(*args, eps, hp, op, *size, _stream(dev))
    if st != OK:
        _raise(st, "m2rnn_add_rmsnorm")
    return out, h


def _scales(like, shape, scales, dev):
    """The scales of a tensor of this shape, new ones when they are not given, and their address."""
    blocks = (*shape[:-1], _blocks(shape[-1]))
    if scales is None:
        scales = torch.empty(blocks, dtype=E8M0, device=like.device)
        return scales, scales.data_ptr()
    return scales, _ptr(scales, "scales", E8M0, blocks, dev)


@_on_stream
def add_rmsnorm_fp8(x, residual, w, eps=1e-5, out=None, scales=None, h=None):
    """``add_rmsnorm`` with its result in 8 bits, for ``linear_fp8``.  Returns (out [..., D] float8_e4m3fn,
    scales [..., ceil(D / 128)] float8_e8m0fnu, h)."""
    dev, h, size, args, hp = _norm_args(x, residual, w, h)
    shape = x.shape
    if out is None:
        out, op, row = _new_bytes(x, shape)
    else:
        op, row = _byte_rows(out, "out", shape, dev)
    scales, sp = _scales(x, shape, scales, dev)
    st = load_library().m2rnn_add_rmsnorm_fp8(*args, eps, hp, op, row, sp, *size, _stream(dev))
    if st != OK:
        _raise(st, "m2rnn_add_rmsnorm_fp8")
    return out, scales, h


@_on_stream
def add_rmsnorm_backward(h, w, dout, dh=None, eps=1e-5, grads=None, workspace=None):
    """Gradients of ``add_rmsnorm`` from its h: dout [..., D] bf16 the gradient of out, dh (of h's type,
    optional) the one that reaches h by the stream.  Returns a dict dx [..., D] bf16, dresidual [..., D] of h's
    type (the same tensor as dx for a bf16 stream), dw [D] float32 (``grads`` may supply any of them
    preallocated)."""
    dev = _device(h)
    shape, kind = h.shape, h.dtype
    D = shape[-1]
    _sizes(D)
    if kind not in (F32, BF16):
        raise TypeError(f"h: expected {F32} or {BF16}, got {kind}")
    hp = _ptr(h, "h", kind, shape, dev)
    g = dict(grads) if grads else {}
    if g.get("dx") is None:
        g["dx"] = _dense(h, BF16)
        dx = g["dx"].data_ptr()
    else:
        dx = _ptr(g["dx"], "dx", BF16, shape, dev)
    if g.get("dresidual") is None:
        g["dresidual"] = g["dx"] if kind is BF16 else _dense(h, kind)
        dr = g["dresidual"].data_ptr()
    else:
        dr = _ptr(g["dresidual"], "dresidual", kind, shape, dev)
    if g.get("dw") is None:
        g["dw"] = torch.empty(D, dtype=F32, device=h.device)
        dw = g["dw"].data_ptr()
    else:
        dw = _ptr(g["dw"], "dw", F32, (D,), dev)
    rows = h.numel() // D if D else 0
    lib = load_library()
    ws, wp, wb = _workspace(workspace, lib.m2rnn_add_rmsnorm_backward_workspace_bytes(rows, D), h)
    st = lib.m2rnn_add_rmsnorm_backward(
        hp, kind is F32, _ptr(w, "w", F32, (D,), dev), eps, _ptr(dout, "dout", BF16, shape, dev),
        _ptr(dh, "dh", kind, shape, dev), dx, None if dr == dx else dr, dw, rows, D, wp, wb, _stream(dev))
    if st != OK:
        _raise(st, "m2rnn_add_rmsnorm_backward")
    return g


# ---------------------------------------------------------------- 8-bit projections
def _source(x, name):
    if x.dtype not in (F32, BF16):
        raise TypeError(f"{name}: expected {F32} or {BF16}, got {x.dtype}")
    return x.dtype is F32


@_on_stream
def quantise_fp8(x, out=None, scales=None):
    """x [..., D] bf16 or float32 in 8 bits with a scale for each 128 channels: (out [..., D]
    float8_e4m3fn, scales [..., ceil(D / 128)] float8_e8m0fnu)."""
    dev, shape, f32 = _device(x), x.shape, _source(x, "x")
    D = shape[-1]
    _sizes(D)
    xp, row = _rows(x, "x", x.dtype, shape, dev)
    if out is None:
        out, op, q_row = _new_bytes(x, shape)
    else:
        op, q_row = _byte_rows(out, "out", shape, dev)
    scales, sp = _scales(x, shape, scales, dev)
    st = load_library().m2rnn_quantise_fp8(xp, f32, row, op, q_row, sp, x.numel() // D if D else 0, D, _stream(dev))
    if st != OK:
        _raise(st, "m2rnn_quantise_fp8")
    return out, scales


@_on_stream
def quantise_weight_fp8(w, out=None, scales=None):
    """A projection's weight w [N, K] (out, in) bf16 or float32 in 8 bits with a scale for each 128 x 128:
    (out [N, K] float8_e4m3fn, scales [ceil(N / 128), ceil(K / 128)] float8_e8m0fnu)."""
    dev, f32 = _device(w), _source(w, "w")
    N, K = shape = w.shape
    _sizes(N, K)
    wp, row = _rows(w, "w", w.dtype, shape, dev)
    if out is None:
        out, op, q_row = _new_bytes(w, shape)
    else:
        op, q_row = _byte_rows(out, "out", shape, dev)
    scales, sp = _scales(w, (_blocks(N), K), scales, dev)
    st = load_library().m2rnn_quantise_weight_fp8(wp, f32, row, op, q_row, sp, N, K, _stream(dev))
    if st != OK:
        _raise(st, "m2rnn_quantise_weight_fp8")
    return out, scales


@_on_stream
def linear_fp8(x, x_scales, w, w_scales, out=None, out_dtype=BF16, workspace=None):
    """Projection in 8 bits: out = x w^T with float32 sums.  x [..., K] and x_scales from
    ``add_rmsnorm_fp8`` or ``quantise_fp8``, or x bf16 or float32 with x_scales None (quantised here, the same
    values); w [N, K] and w_scales from ``quantise_weight_fp8``.  For serving: it has no gradient.  Returns out
    [..., N], bf16 or float32."""
    dev = _device(x)
    shape = x.shape
    K = shape[-1]
    N = w.shape[0]
    _sizes(N, K)
    wp, w_row = _byte_rows(w, "w", (N, K), dev)
    ws = _ptr(w_scales, "w_scales", E8M0, (_blocks(N), _blocks(K)), dev)
    to, kind = (*shape[:-1], N), out_dtype if out is None else out.dtype
    if kind is not BF16 and kind is not F32:
        raise TypeError(f"out: expected {F32} or {BF16}, got {kind}")
    if out is None:
        out = torch.empty(to, dtype=kind, device=x.device)
        op = out.data_ptr()
    else:
        op = _ptr(out, "out", kind, to, dev)
    M = x.numel() // K if K else 0
    lib = load_library()
    if x_scales is None:
        f32 = _source(x, "x")
        xp, row = _rows(x, "x", x.dtype, shape, dev)
        space, sp, sb = _workspace(workspace, lib.m2rnn_linear_quantise_workspace_bytes(f32, M, K), x)
        st = lib.m2rnn_linear_quantise_fp8(xp, f32, row, wp, w_row, ws, op, kind is F32, M, N, K, sp, sb, _stream(dev))
    else:
        xp, row = _byte_rows(x, "x", shape, dev)
        sp = _ptr(x_scales, "x_scales", E8M0, (*shape[:-1], _blocks(K)), dev)
        st = lib.m2rnn_linear_fp8(xp, row, sp, wp, w_row, ws, op, kind is F32, M, N, K, _stream(dev))
    if st != OK:
        _raise(st, "m2rnn_linear_fp8")
    return out


# ---------------------------------------------------------------- gradients
_IS_F32 = {F32: 1, BF16: 0}


def _gradients(grads, out, max_norm, norm, workspace):
    names = grads if isinstance(grads, dict) else None
    grads = list(grads.values()) if names is not None else list(grads)
    if not grads:
        raise ValueError("grads: at least one tensor")
    dev = _device(grads[0])
    # A pass over all tensors for each attribute: a fifth less than one loop's statements.
    n = len(grads)
    kinds = [_IS_F32.get(t.dtype) for t in grads]
    if None in kinds or {t.get_device() for t in grads} != {dev} or not all([t.is_contiguous() for t in grads]):
        for i, t in enumerate(grads):
            if t.dtype not in _IS_F32:
                raise TypeError(f"grads[{i}]: expected {F32} or {BF16}, got {t.dtype}")
            if t.get_device() != dev or not t.is_contiguous():
                _refuse(t, f"grads[{i}]", t.dtype, t.shape, dev)
    ptrs = array("Q", [t.data_ptr() for t in grads])
    sizes = array("q", [t.numel() for t in grads])
    kinds = array("B", kinds)
    if out is None:
        to = ptrs
    elif out is _NORM_ONLY:
        to = None
    else:
        if isinstance(out, dict) and names is not None:
            if out.keys() != names.keys():
                raise ValueError(f"out: {sorted(out.keys() ^ names.keys(), key=str)} on one side only")
            out = [out[name] for name in names]
        else:
            out = list(out.values()) if isinstance(out, dict) else list(out)
        if len(out) != n:
            raise ValueError(f"out: {len(out)} tensors for {n} gradients")
        to = array("Q", [_ptr(o, "out", t.dtype, t.shape, dev) for o, t in zip(out, grads)])
    if norm is None:
        norm = torch.empty((), dtype=F32, device=grads[0].device)
        to_norm = norm.data_ptr()
    else:
        to_norm = _ptr(norm, "norm", F32, (), dev)
    lib = load_library()
    ws, wp, wb = _workspace(workspace, lib.m2rnn_grad_norm_workspace_bytes(n), grads[0])
    st = lib.m2rnn_clip_grad_norm(ptrs.buffer_info()[0], None if to is None else to.buffer_info()[0],
                                  sizes.buffer_info()[0], kinds.buffer_info()[0], n, max_norm,
                                  to_norm, wp, wb, _stream(dev))
    if st != OK:
        _raise(st, "m2rnn_clip_grad_norm")
    return norm


_NORM_ONLY = object()


@_on_stream
def grad_norm(grads, norm=None, workspace=None):
    """The norm of all values of grads (a sequence or dict of contiguous float32 and bf16 tensors)
    together: a float32 scalar on the device."""
    return _gradients(grads, _NORM_ONLY, 0.0, norm, workspace)


@_on_stream
def clip_grad_norm(grads, max_norm, out=None, norm=None, workspace=None):
    """Scales grads (a sequence or dict of contiguous float32 and bf16 tensors, none of which share memory)
    by min(1, max_norm / norm), in place, or into the tensors ``out`` (in the same order; where both are dicts,
    those of the same names).  Returns the norm before that, a float32 scalar on the device.  Where a value is
    infinite or NaN the norm is, and nothing is scaled."""
    return _gradients(grads, out, max_norm, norm, workspace)
