"""Binding of the selective state space block: the short causal convolution with its carried
window, the selective scan and the gated group norm (see include/m2rnn.h for the formulas).

As in the rest of the package, the functions check and marshal arguments, allocate outputs and
workspaces as torch memory when they are not given, and run on the current CUDA stream unless
the keyword ``stream`` names another.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from .m2rnn import OK, M2RNNError, _check, _ptr, _stream_ptr, load_library

BF16, F32 = torch.bfloat16, torch.float32


def _on_stream(f):
    """Adds the keyword ``stream``: the call, and the memory it allocates, belong to it."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        with torch.cuda.stream(stream):
            return f(*args, **kw)
    return call


def _cuda(t):
    if t.device.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    return t.device


def _raise_on(st, where):
    if st != OK:
        raise M2RNNError(st, where)


def _check_tokens(t, name, shape, dev):
    """A bf16 operand [B, T, ...] whose batch and token strides are free: a token's channels
    are contiguous.  Returns the (batch, token) strides in elements."""
    if t.dtype != BF16:
        raise TypeError(f"{name}: expected {BF16}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name}: expected device {dev}, got {t.device}")
    strides, width = t.stride(), 1
    for i in range(len(shape) - 1, 1, -1):
        if strides[i] != width and shape[i] != 1 and t.numel():
            raise ValueError(f"{name}: the channels of a token must be contiguous")
        width *= shape[i]
    return strides[0], strides[1]


def _given(t, name, dtype, shape, dev):
    """``t`` checked, or a new tensor."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _check(t, name, dtype, shape, dev)
    return t


def _workspace(ws, nbytes, dev):
    """The caller's workspace, or a new one; its pointer and size in bytes."""
    if ws is None:
        if nbytes == 0:
            return None, 0, None
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    elif ws.device != dev or not ws.is_contiguous():
        raise ValueError("workspace: must be contiguous and on the inputs' device")
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


# ---------------------------------------------------------------- short causal convolution
def _conv_args(x, w, bias, window):
    dev = _cuda(x)
    B, T, C = x.shape
    sx = _check_tokens(x, "x", (B, T, C), dev)
    _check(w, "w", F32, (C, 4), dev)
    _check(bias, "bias", F32, (C,), dev)
    _check(window, "window", BF16, (B, 3, C), dev)
    return dev, B, T, C, sx


@_on_stream
def conv_silu_window(x, w, bias=None, window=None, out=None, window_out=None):
    """``conv_silu`` continuing an earlier call: x [B, T, C] bf16 (batch and token strides
    free), w [C, 4] and bias [C] float32, window [B, 3, C] bf16 the last three inputs before
    x, oldest first (None: zeros).  Returns (out [B, T, C] bf16, window_out [B, 3, C]), the
    window after x (may be ``window`` itself: in place)."""
    dev, B, T, C, sx = _conv_args(x, w, bias, window)
    out = _given(out, "out", BF16, (B, T, C), dev)
    window_out = _given(window_out, "window_out", BF16, (B, 3, C), dev)
    st = load_library().m2rnn_conv_silu_window_bf16(
        _ptr(x), _ptr(w), _ptr(bias), _ptr(window), _ptr(out), _ptr(window_out), B, T, C, *sx,
        _stream_ptr(None))
    _raise_on(st, "m2rnn_conv_silu_window_bf16")
    return out, window_out


@_on_stream
def conv_silu_step(x, w, bias, window, window_out=None, out=None):
    """One token: x [B, C] bf16, window [B, 3, C] bf16, updated in place unless ``window_out``
    is given.  Returns (out [B, C] bf16, window_out)."""
    B, C = x.shape
    if out is not None:
        _check(out, "out", BF16, (B, C), x.device)
        out = out.unsqueeze(1)
    out, window_out = conv_silu_window(x.unsqueeze(1), w, bias, window, out,
                                       window if window_out is None else window_out)
    return out.squeeze(1), window_out


@_on_stream
def conv_silu_backward(x, w, bias, dout, window=None, grads=None, workspace=None):
    """Gradients of ``conv_silu_window``'s out: dict dx [B, T, C] bf16, dw [C, 4] and dbias [C]
    float32, dwindow [B, 3, C] bf16 (``grads`` may supply any of them preallocated)."""
    dev, B, T, C, sx = _conv_args(x, w, bias, window)
    _check(dout, "dout", BF16, (B, T, C), dev)
    g = dict(grads or {})
    for name, dt, shape in (("dx", BF16, (B, T, C)), ("dw", F32, (C, 4)), ("dbias", F32, (C,)),
                            ("dwindow", BF16, (B, 3, C))):
        g[name] = _given(g.get(name), name, dt, shape, dev)
    lib = load_library()
    wp, wb, ws = _workspace(workspace, lib.m2rnn_conv_silu_backward_workspace_bytes(B, T, C), dev)
    st = lib.m2rnn_conv_silu_backward_bf16(
        _ptr(x), _ptr(w), _ptr(bias), _ptr(window), _ptr(dout), _ptr(g["dx"]), _ptr(g["dw"]),
        _ptr(g["dbias"]), _ptr(g["dwindow"]), B, T, C, *sx, wp, wb, _stream_ptr(None))
    _raise_on(st, "m2rnn_conv_silu_backward_bf16")
    return g


# ---------------------------------------------------------------- selective scan
def _ssm_args(inputs):
    """Checks the scan's inputs; (device, sizes, pointers of q..w_r, strides array)."""
    q, k, v, a = (inputs[n] for n in ("q", "k", "v", "a"))
    dev = _cuda(q)
    B, T, G, K = q.shape
    N, V = v.shape[2:]
    if G < 1 or N % G:
        raise ValueError(f"q, k must have a number of heads that divides {N}, got {G}")
    strides = (ctypes.c_longlong * 8)(
        *_check_tokens(q, "q", (B, T, G, K), dev), *_check_tokens(k, "k", (B, T, G, K), dev),
        *_check_tokens(v, "v", (B, T, N, V), dev), *_check_tokens(a, "a", (B, T, N), dev))
    alpha, beta, w_r = (inputs[n] for n in ("alpha", "beta", "w_r"))
    _check(alpha, "alpha", F32, (N,), dev)
    _check(beta, "beta", F32, (N,), dev)
    _check(w_r, "w_r", F32, (N, V), dev)
    return dev, (B, T, N, G, K, V), [_ptr(t) for t in (q, k, v, a, alpha, beta, w_r)], strides


def ssm_states_bytes(B, T, N, K, V) -> int:
    return int(load_library().m2rnn_ssm_states_bytes(B, T, N, K, V))


def ssm_workspace_bytes(B, T, N, Nqk, K, V, backward=False) -> int:
    return int(load_library().m2rnn_ssm_workspace_bytes(B, T, N, Nqk, K, V, int(backward)))


def _ssm_run(inputs, y, H_T, Hs, workspace):
    dev, sizes, ptrs, strides = _ssm_args(inputs)
    B, T, N, G, K, V = sizes
    H0 = inputs.get("H0")
    _check(H0, "H0", F32, (B, N, K, V), dev)
    y = _given(y, "y", BF16, (B, T, N, V), dev)
    H_T = _given(H_T, "H_T", F32, (B, N, K, V), dev)
    lib = load_library()
    wp, wb, ws = _workspace(workspace, lib.m2rnn_ssm_workspace_bytes(*sizes, 0), dev)
    st = lib.m2rnn_ssm_forward_bf16(*ptrs, _ptr(H0), _ptr(y), _ptr(H_T), _ptr(Hs), strides,
                                    *sizes, wp, wb, _stream_ptr(None))
    _raise_on(st, "m2rnn_ssm_forward_bf16")
    return y, H_T


@_on_stream
def ssm_forward(inputs: dict, y=None, H_T=None, workspace=None):
    """Selective scan of a prompt: inputs q, k [B, T, Nqk, K], v [B, T, N, V], a [B, T, N] bf16
    (batch and token strides free, Nqk divides N), alpha, beta [N], w_r [N, V] float32 and
    optionally H0 [B, N, K, V] float32.  Returns (y [B, T, N, V] bf16, H_T float32)."""
    return _ssm_run(inputs, y, H_T, None, workspace)


@_on_stream
def ssm_forward_train(inputs: dict, y=None, H_T=None, Hs=None, workspace=None):
    """``ssm_forward`` that also keeps the states the backward reads.  Returns (y, H_T, Hs)."""
    q, v = inputs["q"], inputs["v"]
    nbytes = ssm_states_bytes(q.shape[0], q.shape[1], v.shape[2], q.shape[3], v.shape[3])
    if Hs is None:
        Hs = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    _check(Hs, "Hs", torch.uint8, (nbytes,), q.device)
    y, H_T = _ssm_run(inputs, y, H_T, Hs, workspace)
    return y, H_T, Hs


@_on_stream
def ssm_backward(inputs: dict, Hs, dy, dH_T=None, grads=None, workspace=None):
    """Gradients of a loss through y (dy [B, T, N, V] bf16) and H_T (dH_T float32, optional),
    with Hs of ``ssm_forward_train`` on the same inputs.  Returns a dict dq, dk, dv, da (bf16),
    dalpha, dbeta, dw_r, dH0 (float32; ``grads`` may supply any of them preallocated)."""
    dev, sizes, ptrs, strides = _ssm_args(inputs)
    B, T, N, G, K, V = sizes
    lib = load_library()
    _check(Hs, "Hs", torch.uint8, (lib.m2rnn_ssm_states_bytes(B, T, N, K, V),), dev)
    _check(dy, "dy", BF16, (B, T, N, V), dev)
    _check(dH_T, "dH_T", F32, (B, N, K, V), dev)
    g = dict(grads or {})
    shapes = {"dq": (BF16, (B, T, G, K)), "dk": (BF16, (B, T, G, K)), "dv": (BF16, (B, T, N, V)),
              "da": (BF16, (B, T, N)), "dalpha": (F32, (N,)), "dbeta": (F32, (N,)),
              "dw_r": (F32, (N, V)), "dH0": (F32, (B, N, K, V))}
    for name, (dt, shape) in shapes.items():
        g[name] = _given(g.get(name), name, dt, shape, dev)
    wp, wb, ws = _workspace(workspace, lib.m2rnn_ssm_workspace_bytes(*sizes, 1), dev)
    st = lib.m2rnn_ssm_backward_bf16(*ptrs, _ptr(Hs), _ptr(dy), _ptr(dH_T),
                                     *[_ptr(g[n]) for n in shapes], strides, *sizes, wp, wb,
                                     _stream_ptr(None))
    _raise_on(st, "m2rnn_ssm_backward_bf16")
    return g


@_on_stream
def ssm_step(q, k, v, a, alpha, beta, w_r, H_in, H_out=None, y=None):
    """One token of the scan: q, k [B, Nqk, K], v [B, N, V], a [B, N] bf16, H_in [B, N, K, V]
    float32 (None: zero).  Writes H_out (H_in itself when not given: in place) and
    y [B, N, V] bf16; returns (y, H_out)."""
    dev = _cuda(q)
    B, G, K = q.shape
    N, V = v.shape[1:]
    if G < 1 or N % G:
        raise ValueError(f"q, k must have a number of heads that divides {N}, got {G}")
    for t, name, dt, shape in ((q, "q", BF16, (B, G, K)), (k, "k", BF16, (B, G, K)),
                               (v, "v", BF16, (B, N, V)), (a, "a", BF16, (B, N)),
                               (alpha, "alpha", F32, (N,)), (beta, "beta", F32, (N,)),
                               (w_r, "w_r", F32, (N, V)), (H_in, "H_in", F32, (B, N, K, V))):
        _check(t, name, dt, shape, dev)
    H_out = _given(H_in if H_out is None else H_out, "H_out", F32, (B, N, K, V), dev)
    y = _given(y, "y", BF16, (B, N, V), dev)
    st = load_library().m2rnn_ssm_step_bf16(
        *[_ptr(t) for t in (q, k, v, a, alpha, beta, w_r, H_in, H_out, y)], B, N, G, K, V,
        _stream_ptr(None))
    _raise_on(st, "m2rnn_ssm_step_bf16")
    return y, H_out


# ---------------------------------------------------------------- gated group norm
def _norm_args(y, g_pre, w, bias, groups):
    dev = _cuda(y)
    D = y.shape[-1]
    if y.dtype not in (F32, BF16):
        raise TypeError(f"y: expected {F32} or {BF16}, got {y.dtype}")
    if groups < 1 or D % groups:
        raise ValueError(f"groups: {groups} does not divide the {D} channels")
    _check(y, "y", y.dtype, y.shape, dev)
    _check(g_pre, "g_pre", BF16, y.shape, dev)
    _check(w, "w", F32, (D,), dev)
    _check(bias, "bias", F32, (D,), dev)
    return dev, D, y.numel() // D if D else 0


@_on_stream
def gate_groupnorm(y, g_pre, w, bias=None, groups=1, eps=1e-5, out=None):
    """Group norm over the last axis of y [..., D] (float32 or bf16) in ``groups`` groups, with
    w, bias [D] float32, times SiLU(g_pre) (g_pre [..., D] bf16); with g_pre None, SiLU of the
    norm itself.  Returns out [..., D] bf16."""
    dev, D, rows = _norm_args(y, g_pre, w, bias, groups)
    out = _given(out, "out", BF16, y.shape, dev)
    st = load_library().m2rnn_gate_groupnorm(
        _ptr(y), int(y.dtype == F32), _ptr(g_pre), _ptr(w), _ptr(bias), float(eps), _ptr(out),
        rows, D, groups, _stream_ptr(None))
    _raise_on(st, "m2rnn_gate_groupnorm")
    return out


@_on_stream
def gate_groupnorm_backward(y, g_pre, w, bias, dout, groups=1, eps=1e-5, grads=None,
                            workspace=None):
    """Gradients of ``gate_groupnorm``: dict dy (of y's type), dg_pre (bf16, None without
    g_pre), dw, dbias [D] float32 (``grads`` may supply any of them preallocated)."""
    dev, D, rows = _norm_args(y, g_pre, w, bias, groups)
    _check(dout, "dout", BF16, y.shape, dev)
    g = dict(grads or {})
    for name, dt, shape in (("dy", y.dtype, y.shape), ("dg_pre", BF16, y.shape),
                            ("dw", F32, (D,)), ("dbias", F32, (D,))):
        g[name] = None if name == "dg_pre" and g_pre is None else _given(g.get(name), name, dt,
                                                                         shape, dev)
    lib = load_library()
    wp, wb, ws = _workspace(
        workspace, lib.m2rnn_gate_groupnorm_backward_workspace_bytes(rows, D, groups), dev)
    st = lib.m2rnn_gate_groupnorm_backward(
        _ptr(y), int(y.dtype == F32), _ptr(g_pre), _ptr(w), _ptr(bias), float(eps), _ptr(dout),
        _ptr(g["dy"]), _ptr(g["dg_pre"]), _ptr(g["dw"]), _ptr(g["dbias"]), rows, D, groups, wp,
        wb, _stream_ptr(None))
    _raise_on(st, "m2rnn_gate_groupnorm_backward")
    return g
