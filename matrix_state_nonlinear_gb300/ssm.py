"""Binding of the selective state space block: the short causal convolution with its carried
window, the selective scan and the gated group norm (see include/m2rnn.h for the formulas).

As in the rest of the package, the functions check and marshal arguments, allocate outputs and
workspaces as torch memory when they are not given, and run on the current CUDA stream unless
the keyword ``stream`` names another.  The tensors have to be on the current device (the stream's
device, where one is named).  A token's kernels take a few microseconds, so the checks
are one pass over each tensor's attributes and the error messages are made only on failure.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from .m2rnn import OK, M2RNNError, load_library

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def _on_stream(f):
    """Adds the keyword ``stream``: the call, and the memory it allocates, belong to it."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        with torch.cuda.stream(stream):
            return f(*args, **kw)
    return call


def _device(t):
    """The CUDA device index of a tensor; refuses host tensors, and tensors of another device than
    the current one, on which the kernels would launch."""
    if not t.is_cuda:
        raise ValueError("inputs must be CUDA tensors")
    dev, current = t.get_device(), torch._C._cuda_getDevice()
    if dev != current:
        raise ValueError(f"inputs are on cuda:{dev}, the current device is cuda:{current}")
    return dev


def _refuse(t, name, dtype, shape, dev):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name}: expected device cuda:{dev}, got {t.device}")
    raise ValueError(f"{name}: must be contiguous")


def _ptr(t, name, dtype, shape, dev):
    """The address of a tensor of this type and shape, dense and on this device; None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _refuse(t, name, dtype, shape, dev)
    return t.data_ptr()


def _tokens(t, name, shape, dev):
    """A bf16 operand [B, T, ...] whose batch and token strides are free: a token's channels are
    contiguous.  Returns (address, batch stride, token stride), strides in elements."""
    if t.dtype is not BF16 or t.shape != shape or t.get_device() != dev:
        _refuse(t, name, BF16, shape, dev)
    s = t.stride()
    if t.numel():
        width = 1
        for i in range(len(shape) - 1, 1, -1):
            if s[i] != width and shape[i] != 1:
                raise ValueError(f"{name}: the channels of a token must be contiguous")
            width *= shape[i]
    return t.data_ptr(), s[0], s[1]


def _stream(dev):
    return torch._C._cuda_getCurrentRawStream(dev)


def _workspace(ws, nbytes, like):
    """The caller's workspace, or a new one beside ``like``: (tensor, address, bytes)."""
    if ws is None:
        if nbytes == 0:
            return None, None, 0
        ws = torch.empty(nbytes, dtype=U8, device=like.device)
    elif ws.get_device() != like.get_device() or not ws.is_contiguous():
        raise ValueError("workspace: must be contiguous and on the inputs' device")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _raise(st, where):
    raise M2RNNError(st, where)


def _sizes(*n):
    """Sizes that the library takes as 32-bit integers; ctypes would cut larger ones down."""
    if max(n) > 0x7fffffff:
        raise ValueError(f"sizes of 2^31 and above are not supported: {n}")
    return n


# ---------------------------------------------------------------- short causal convolution
def _taps(w, C, dev):
    p = _ptr(w, "w", F32, (C, 4), dev)
    if p is not None and p % 16:
        raise ValueError("w: must be 16-byte aligned (a view into a larger buffer may not be; copy it once)")
    return p


@_on_stream
def conv_silu_window(x, w, bias=None, window=None, out=None, window_out=None):
    """``conv_silu`` continuing an earlier call: x [B, T, C] bf16 (batch and token strides
    free), w [C, 4] (16-byte aligned) and bias [C] float32, window [B, 3, C] bf16 the last three
    inputs before x, oldest first (None: zeros).  Returns (out [B, T, C] bf16, window_out
    [B, 3, C]), the window after x (may be ``window`` itself: in place)."""
    dev = _device(x)
    B, T, C = shape = x.shape
    _sizes(B, T, C)
    xp, xb, xt = _tokens(x, "x", shape, dev)
    if out is None:
        out = x.new_empty(shape)
    if window_out is None:
        window_out = x.new_empty((B, 3, C))
    st = load_library().m2rnn_conv_silu_window_bf16(
        xp, _taps(w, C, dev), _ptr(bias, "bias", F32, (C,), dev),
        _ptr(window, "window", BF16, (B, 3, C), dev), _ptr(out, "out", BF16, shape, dev),
        _ptr(window_out, "window_out", BF16, (B, 3, C), dev), B, T, C, xb, xt, _stream(dev))
    if st != OK:
        _raise(st, "m2rnn_conv_silu_window_bf16")
    return out, window_out


@_on_stream
def conv_silu_step(x, w, bias, window, window_out=None, out=None):
    """One token: x [B, C] bf16 (batch stride free), window [B, 3, C] bf16 (None: zeros), updated
    in place unless ``window_out`` is given.  Returns (out [B, C] bf16, window_out)."""
    dev = _device(x)
    B, C = shape = x.shape
    _sizes(B, C)
    if x.dtype is not BF16 or (x.stride(1) != 1 and C > 1):
        _refuse(x, "x", BF16, shape, dev)
    if out is None:
        out = x.new_empty(shape)
    if window_out is None:
        window_out = x.new_empty((B, 3, C)) if window is None else window
    st = load_library().m2rnn_conv_silu_window_bf16(
        x.data_ptr(), _taps(w, C, dev), _ptr(bias, "bias", F32, (C,), dev),
        _ptr(window, "window", BF16, (B, 3, C), dev), _ptr(out, "out", BF16, shape, dev),
        _ptr(window_out, "window_out", BF16, (B, 3, C), dev), B, 1, C, x.stride(0), C, _stream(dev))
    if st != OK:
        _raise(st, "m2rnn_conv_silu_window_bf16")
    return out, window_out


@_on_stream
def conv_silu_backward(x, w, bias, dout, window=None, grads=None, workspace=None):
    """Gradients of ``conv_silu_window``'s out: dict dx [B, T, C] bf16, dw [C, 4] and dbias [C]
    float32, dwindow [B, 3, C] bf16 (``grads`` may supply any of them preallocated)."""
    dev = _device(x)
    B, T, C = shape = x.shape
    _sizes(B, T, C)
    xp, xb, xt = _tokens(x, "x", shape, dev)
    g = dict(grads or {})
    ptrs = []
    for name, like, size in (("dx", x, shape), ("dw", w, (C, 4)), ("dbias", w, (C,)),
                             ("dwindow", x, (B, 3, C))):
        if g.get(name) is None:
            g[name] = like.new_empty(size)
        ptrs.append(_ptr(g[name], name, BF16 if like is x else F32, size, dev))
    lib = load_library()
    ws, wp, wb = _workspace(workspace, lib.m2rnn_conv_silu_backward_workspace_bytes(B, T, C), x)
    st = lib.m2rnn_conv_silu_backward_bf16(
        xp, _taps(w, C, dev), _ptr(bias, "bias", F32, (C,), dev),
        _ptr(window, "window", BF16, (B, 3, C), dev), _ptr(dout, "dout", BF16, shape, dev), *ptrs,
        B, T, C, xb, xt, wp, wb, _stream(dev))
    if st != OK:
        _raise(st, "m2rnn_conv_silu_backward_bf16")
    return g


# ---------------------------------------------------------------- selective scan
_EIGHT = ctypes.c_longlong * 8


def _ssm_args(inputs):
    """Checks the scan's inputs: (device, sizes, addresses of q .. w_r, strides)."""
    q, k, v, a = inputs["q"], inputs["k"], inputs["v"], inputs["a"]
    dev = _device(q)
    B, T, G, K = shape = q.shape
    N, V = v.shape[2:]
    _sizes(B, T, G, K, N, V)
    if G < 1 or N % G:
        raise ValueError(f"q, k must have a number of heads that divides {N}, got {G}")
    qp, qb, qt = _tokens(q, "q", shape, dev)
    kp, kb, kt = _tokens(k, "k", shape, dev)
    vp, vb, vt = _tokens(v, "v", (B, T, N, V), dev)
    ap, ab, at = _tokens(a, "a", (B, T, N), dev)
    ptrs = (qp, kp, vp, ap, _ptr(inputs["alpha"], "alpha", F32, (N,), dev),
            _ptr(inputs["beta"], "beta", F32, (N,), dev),
            _ptr(inputs["w_r"], "w_r", F32, (N, V), dev))
    return dev, (B, T, N, G, K, V), ptrs, _EIGHT(qb, qt, kb, kt, vb, vt, ab, at)


def ssm_states_bytes(B, T, N, K, V) -> int:
    return int(load_library().m2rnn_ssm_states_bytes(*_sizes(B, T, N, K, V)))


def ssm_workspace_bytes(B, T, N, Nqk, K, V, backward=False) -> int:
    return int(load_library().m2rnn_ssm_workspace_bytes(*_sizes(B, T, N, Nqk, K, V), int(backward)))


def _ssm_run(inputs, y, H_T, Hs, keep, workspace):
    dev, sizes, ptrs, strides = _ssm_args(inputs)
    B, T, N, G, K, V = sizes
    state = (B, N, K, V)
    H0 = inputs.get("H0")
    if y is None:
        y = inputs["v"].new_empty((B, T, N, V))
    if H_T is None:
        H_T = inputs["alpha"].new_empty(state)
    lib = load_library()
    if keep:
        nbytes = lib.m2rnn_ssm_states_bytes(B, T, N, K, V)
        if Hs is None:
            Hs = torch.empty(nbytes, dtype=U8, device=y.device)
        kept = _ptr(Hs, "Hs", U8, (nbytes,), dev)
    else:
        kept = None
    ws, wp, wb = _workspace(workspace, lib.m2rnn_ssm_workspace_bytes(*sizes, 0), y)
    st = lib.m2rnn_ssm_forward_bf16(
        *ptrs, _ptr(H0, "H0", F32, state, dev), _ptr(y, "y", BF16, (B, T, N, V), dev),
        _ptr(H_T, "H_T", F32, state, dev), kept, strides, *sizes, wp, wb, _stream(dev))
    if st != OK:
        _raise(st, "m2rnn_ssm_forward_bf16")
    return y, H_T, Hs


@_on_stream
def ssm_forward(inputs: dict, y=None, H_T=None, workspace=None):
    """Selective scan of a prompt: inputs q, k [B, T, Nqk, K], v [B, T, N, V], a [B, T, N] bf16
    (batch and token strides free, Nqk divides N), alpha, beta [N], w_r [N, V] float32 and
    optionally H0 [B, N, K, V] float32.  Returns (y [B, T, N, V] bf16, H_T float32)."""
    return _ssm_run(inputs, y, H_T, None, False, workspace)[:2]


@_on_stream
def ssm_forward_train(inputs: dict, y=None, H_T=None, Hs=None, workspace=None):
    """``ssm_forward`` that also keeps the states the backward reads.  Returns (y, H_T, Hs)."""
    return _ssm_run(inputs, y, H_T, Hs, True, workspace)


@_on_stream
def ssm_backward(inputs: dict, Hs, dy, dH_T=None, grads=None, workspace=None):
    """Gradients of a loss through y (dy [B, T, N, V] bf16) and H_T (dH_T float32, optional),
    with Hs of ``ssm_forward_train`` on the same inputs.  Returns a dict dq, dk, dv, da (bf16),
    dalpha, dbeta, dw_r, dH0 (float32; ``grads`` may supply any of them preallocated)."""
    dev, sizes, ptrs, strides = _ssm_args(inputs)
    B, T, N, G, K, V = sizes
    lib = load_library()
    g = dict(grads or {})
    alpha = inputs["alpha"]
    out = []
    for name, like, shape in (("dq", dy, (B, T, G, K)), ("dk", dy, (B, T, G, K)),
                              ("dv", dy, (B, T, N, V)), ("da", dy, (B, T, N)),
                              ("dalpha", alpha, (N,)), ("dbeta", alpha, (N,)),
                              ("dw_r", alpha, (N, V)), ("dH0", alpha, (B, N, K, V))):
        if g.get(name) is None:
            g[name] = like.new_empty(shape)
        out.append(_ptr(g[name], name, BF16 if like is dy else F32, shape, dev))
    ws, wp, wb = _workspace(workspace, lib.m2rnn_ssm_workspace_bytes(*sizes, 1), alpha)
    st = lib.m2rnn_ssm_backward_bf16(
        *ptrs, _ptr(Hs, "Hs", U8, (lib.m2rnn_ssm_states_bytes(B, T, N, K, V),), dev),
        _ptr(dy, "dy", BF16, (B, T, N, V), dev), _ptr(dH_T, "dH_T", F32, (B, N, K, V), dev), *out,
        strides, *sizes, wp, wb, _stream(dev))
    if st != OK:
        _raise(st, "m2rnn_ssm_backward_bf16")
    return g


@_on_stream
def ssm_step(q, k, v, a, alpha, beta, w_r, H_in, H_out=None, y=None):
    """One token of the scan: q, k [B, Nqk, K], v [B, N, V], a [B, N] bf16, H_in [B, N, K, V]
    float32 (None: zero).  Writes H_out (H_in itself when not given: in place) and
    y [B, N, V] bf16; returns (y, H_out)."""
    dev = _device(q)
    B, G, K = q.shape
    N, V = v.shape[1:]
    _sizes(B, G, K, N, V)
    if G < 1 or N % G:
        raise ValueError(f"q, k must have a number of heads that divides {N}, got {G}")
    state = (B, N, K, V)
    if H_out is None:
        H_out = alpha.new_empty(state) if H_in is None else H_in
    if y is None:
        y = v.new_empty((B, N, V))
    st = load_library().m2rnn_ssm_step_bf16(
        _ptr(q, "q", BF16, (B, G, K), dev), _ptr(k, "k", BF16, (B, G, K), dev),
        _ptr(v, "v", BF16, (B, N, V), dev), _ptr(a, "a", BF16, (B, N), dev),
        _ptr(alpha, "alpha", F32, (N,), dev), _ptr(beta, "beta", F32, (N,), dev),
        _ptr(w_r, "w_r", F32, (N, V), dev), _ptr(H_in, "H_in", F32, state, dev),
        _ptr(H_out, "H_out", F32, state, dev), _ptr(y, "y", BF16, (B, N, V), dev), B, N, G, K, V,
        _stream(dev))
    if st != OK:
        _raise(st, "m2rnn_ssm_step_bf16")
    return y, H_out


# ---------------------------------------------------------------- gated group norm
def _norm_args(y, g_pre, w, bias, groups):
    """Checks the norm's inputs: (device, channels, rows, addresses of y, its type, g_pre, w, bias)."""
    dev = _device(y)
    shape = y.shape
    D = shape[-1]
    _sizes(D, groups)
    if y.dtype not in (F32, BF16):
        raise TypeError(f"y: expected {F32} or {BF16}, got {y.dtype}")
    if groups < 1 or D % groups:
        raise ValueError(f"groups: {groups} does not divide the {D} channels")
    return dev, D, y.numel() // D if D else 0, (
        _ptr(y, "y", y.dtype, shape, dev), int(y.dtype is F32), _ptr(g_pre, "g_pre", BF16, shape, dev),
        _ptr(w, "w", F32, (D,), dev), _ptr(bias, "bias", F32, (D,), dev))


@_on_stream
def gate_groupnorm(y, g_pre, w, bias=None, groups=1, eps=1e-5, out=None):
    """Group norm over the last axis of y [..., D] (float32 or bf16) in ``groups`` groups, with
    w, bias [D] float32, times SiLU(g_pre) (g_pre [..., D] bf16); with g_pre None, SiLU of the
    norm itself.  Returns out [..., D] bf16."""
    dev, D, rows, args = _norm_args(y, g_pre, w, bias, groups)
    if out is None:
        out = torch.empty_like(y, dtype=BF16)
    st = load_library().m2rnn_gate_groupnorm(*args, eps, _ptr(out, "out", BF16, y.shape, dev), rows,
                                             D, groups, _stream(dev))
    if st != OK:
        _raise(st, "m2rnn_gate_groupnorm")
    return out


@_on_stream
def gate_groupnorm_backward(y, g_pre, w, bias, dout, groups=1, eps=1e-5, grads=None,
                            workspace=None):
    """Gradients of ``gate_groupnorm``: dict dy (of y's type), dg_pre (bf16, None without
    g_pre), dw, dbias [D] float32 (``grads`` may supply any of them preallocated)."""
    dev, D, rows, args = _norm_args(y, g_pre, w, bias, groups)
    g = dict(grads or {})
    ptrs = []
    for name, like, shape in (("dy", y, y.shape), ("dg_pre", g_pre, y.shape), ("dw", w, (D,)),
                              ("dbias", w, (D,))):
        if like is None:
            g[name] = None
        elif g.get(name) is None:
            g[name] = like.new_empty(shape)
        ptrs.append(None if like is None else _ptr(g[name], name, like.dtype, shape, dev))
    lib = load_library()
    ws, wp, wb = _workspace(
        workspace, lib.m2rnn_gate_groupnorm_backward_workspace_bytes(rows, D, groups), y)
    st = lib.m2rnn_gate_groupnorm_backward(*args, eps, _ptr(dout, "dout", BF16, y.shape, dev), *ptrs,
                                           rows, D, groups, wp, wb, _stream(dev))
    if st != OK:
        _raise(st, "m2rnn_gate_groupnorm_backward")
    return g
