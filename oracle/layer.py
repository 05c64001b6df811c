"""fp64 oracle of what stands around a block in a stack: the residual RMS norm and its gradients, 8-bit
values with block scales, the product of such values, and the clipping of gradients.  NumPy only; shares
no code with the kernels."""
import math

import numpy as np

BLOCK = 128


def rmsnorm(h, w, eps):
    """h [..., D] (the stream after the addition, as its type holds it) -> out."""
    return h / np.sqrt(np.mean(h * h, -1, keepdims=True) + eps) * w


def rmsnorm_backward(h, w, dout, dh, eps):
    """Gradients (d, dw) of <rmsnorm, dout> + <h, dh>, and the sums of the magnitudes of their terms."""
    D = h.shape[-1]
    r = 1.0 / np.sqrt(np.mean(h * h, -1, keepdims=True) + eps)
    g = dout * w
    shared = h * r ** 3 * np.sum(g * h, -1, keepdims=True) / D
    d = r * g - shared
    size = np.abs(r * g) + np.abs(h) * r ** 3 * np.sum(np.abs(g * h), -1, keepdims=True) / D
    if dh is not None:
        d, size = d + dh, size + np.abs(dh)
    terms = (dout * h * r).reshape(-1, D)
    return d, terms.sum(0), size, np.abs(terms).sum(0)


def scale_of(amax):
    """The least power of two s >= 2^-126 with amax / s <= 448; NaN for an infinite or NaN amax."""
    if not math.isfinite(amax):
        return math.nan
    e = -126
    while math.ldexp(448.0, e) < amax:
        e += 1
    return math.ldexp(1.0, e)


def e4m3(v):
    """The nearest e4m3 value to each of v (|v| <= 448), ties to even."""
    v = np.asarray(v, np.float64)
    with np.errstate(divide="ignore"):
        step = np.exp2(np.maximum(np.floor(np.log2(np.abs(v))), -6.0) - 3.0)
    return np.rint(v / step) * step


def row_scales(x):
    """x [R, D] -> scales [R, blocks]."""
    return np.array([[scale_of(np.max(np.abs(r[c:c + BLOCK]))) for c in range(0, x.shape[1], BLOCK)] for r in x])


def quantise(x):
    """x [R, D] -> (e4m3 values, scales)."""
    s = row_scales(x)
    return e4m3(x / np.repeat(s, BLOCK, 1)[:, :x.shape[1]]), s


def quantise_weight(w):
    """w [N, K] -> (e4m3 values, a scale for each 128 x 128)."""
    N, K = w.shape
    s = np.array([[scale_of(np.max(np.abs(w[n:n + BLOCK, k:k + BLOCK]))) for k in range(0, K, BLOCK)]
                  for n in range(0, N, BLOCK)])
    return e4m3(w / spread(s, N, K)), s


def spread(s, N, K):
    return np.repeat(np.repeat(s, BLOCK, 0)[:N], BLOCK, 1)[:, :K]


def linear(q, s, wq, ws):
    """Values [M, K] and weights [N, K] with their scales -> (out [M, N], the sums of its terms' magnitudes)."""
    x, w = q * np.repeat(s, BLOCK, 1)[:, :q.shape[1]], wq * spread(ws, *wq.shape)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def clip(grads, max_norm):
    """(norm, clipped gradients)."""
    n = math.sqrt(math.fsum(float(np.sum(np.square(g.astype(np.longdouble)))) for g in grads))
    by = max_norm / n if math.isfinite(n) and n > max_norm else 1.0
    return n, [g * by for g in grads]
