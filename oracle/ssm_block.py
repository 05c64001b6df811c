"""fp64 CPU oracle of the selective state space block: short causal convolution with its
carried window, selective scan, gated group norm, and their gradients.  TEST INFRASTRUCTURE
ONLY; written from the formulas, token by token, sharing no code with the CUDA library.

  conv:  pre[t] = bias + sum_j w[j] X[t-3+j], out = SiLU(pre), X = window then x
  scan:  d = softplus(a + beta), f = exp(-alpha d), H_t = f H_{t-1} + d k v^T,
         y = H^T q + w_r v; head n reads head n Nqk / N of q and k
  norm:  n = (y - mean) / sqrt(var + eps) per group, p = w n + b,
         out = p SiLU(g) or SiLU(p)
"""
from __future__ import annotations

import numpy as np


def _sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def _dsilu(x):
    s = _sigmoid(x)
    return s * (1.0 + x * (1.0 - s))


# ---------------------------------------------------------------- convolution
def conv_window(x, w, bias=None, window=None):
    """x [B, T, C], w [C, 4], window [B, 3, C]: (out, window after x, pre, X)."""
    B, T, C = x.shape
    X = np.concatenate([np.zeros((B, 3, C)) if window is None else window, x], 1)
    pre = np.zeros((B, T, C)) + (0.0 if bias is None else bias)
    for t in range(T):
        for j in range(4):
            pre[:, t] += w[:, j] * X[:, t + j]
    return pre * _sigmoid(pre), X[:, T:], pre, X


def conv_window_backward(x, w, bias, dout, window=None):
    B, T, C = x.shape
    _, _, pre, X = conv_window(x, w, bias, window)
    dpre = dout * _dsilu(pre)
    dX, dw = np.zeros_like(X), np.zeros((C, 4))
    for t in range(T):
        for j in range(4):
            dX[:, t + j] += w[:, j] * dpre[:, t]
            dw[:, j] += (dpre[:, t] * X[:, t + j]).sum(0)
    return dict(dx=dX[:, 3:], dw=dw, dbias=dpre.sum((0, 1)), dwindow=dX[:, :3])


# ---------------------------------------------------------------- selective scan
def _gate(a, alpha, beta):
    x = a + beta
    d = np.maximum(x, 0.0) + np.log1p(np.exp(-np.abs(x)))
    return x, d, np.exp(-alpha * d)


def ssm_scan(q, k, v, a, alpha, beta, w_r, H0=None):
    """(y [B, T, N, V], states [T + 1] of [B, N, K, V])."""
    B, T, N, V = v.shape
    G, K = q.shape[2:]
    _, d, f = _gate(a, alpha, beta)
    H = np.zeros((B, N, K, V)) if H0 is None else H0.copy()
    states, y = [H], np.empty((B, T, N, V))
    for t in range(T):
        kt, qt = np.repeat(k[:, t], N // G, 1), np.repeat(q[:, t], N // G, 1)
        H = f[:, t, :, None, None] * H + (d[:, t, :, None] * kt)[..., None] * v[:, t, :, None, :]
        states.append(H)
        y[:, t] = np.einsum("bnkv,bnk->bnv", H, qt) + w_r * v[:, t]
    return y, states


def ssm_backward(q, k, v, a, alpha, beta, w_r, dy, H0=None, dH_T=None, bound=False):
    """Gradients by the reverse scan; with ``bound`` every difference is a sum, so that on
    absolute inputs each result is the sum of its terms' magnitudes."""
    B, T, N, V = v.shape
    G, K = q.shape[2:]
    rep, sign = N // G, 1.0 if bound else -1.0
    x, d, f = _gate(a, alpha, beta)
    _, states = ssm_scan(q, k, v, a, alpha, beta, w_r, H0)
    D = np.zeros((B, N, K, V)) if dH_T is None else dH_T.copy()
    dq, dk = np.zeros((B, T, N, K)), np.zeros((B, T, N, K))
    dv, g, kgv = np.zeros((B, T, N, V)), np.zeros((B, T, N)), np.zeros((B, T, N))
    for t in range(T - 1, -1, -1):
        kt, qt = np.repeat(k[:, t], rep, 1), np.repeat(q[:, t], rep, 1)
        D = D + qt[..., None] * dy[:, t, :, None, :]
        dq[:, t] = np.einsum("bnkv,bnv->bnk", states[t + 1], dy[:, t])
        gv = np.einsum("bnkv,bnv->bnk", D, v[:, t])
        dk[:, t] = d[:, t, :, None] * gv
        kgv[:, t] = (kt * gv).sum(-1)
        dv[:, t] = d[:, t, :, None] * np.einsum("bnkv,bnk->bnv", D, kt) + w_r * dy[:, t]
        g[:, t] = f[:, t] * (D * states[t]).sum((-2, -1))
        D = f[:, t, :, None, None] * D
    da = _sigmoid(x) * (kgv + sign * alpha * g)
    return dict(dq=dq.reshape(B, T, G, rep, K).sum(3), dk=dk.reshape(B, T, G, rep, K).sum(3),
                dv=dv, da=da, dalpha=sign * (d * g).sum((0, 1)), dbeta=da.sum((0, 1)),
                dw_r=(dy * v).sum((0, 1)), dH0=D)


# ---------------------------------------------------------------- gated group norm
def _normalise(y, groups, eps):
    z = y.reshape(y.shape[0], groups, -1)
    z = z - z.mean(-1, keepdims=True)
    inv = 1.0 / np.sqrt((z * z).mean(-1, keepdims=True) + eps)
    return z * inv, inv


def gate_groupnorm(y, g, w, bias, groups, eps):
    n, _ = _normalise(y, groups, eps)
    p = n.reshape(y.shape) * w + (0.0 if bias is None else bias)
    return p * _sigmoid(p) if g is None else p * g * _sigmoid(g)


def gate_groupnorm_backward(y, g, w, bias, dout, groups, eps):
    n, inv = _normalise(y, groups, eps)
    nf = n.reshape(y.shape)
    p = nf * w + (0.0 if bias is None else bias)
    dp = dout * (_dsilu(p) if g is None else g * _sigmoid(g))
    dn = (dp * w).reshape(n.shape)
    dy = inv * (dn - dn.mean(-1, keepdims=True) - n * (dn * n).mean(-1, keepdims=True))
    return dict(dy=dy.reshape(y.shape), dg_pre=None if g is None else dout * p * _dsilu(g),
                dw=(dp * nf).sum(0), dbias=dp.sum(0))
