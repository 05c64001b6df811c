"""The oracle of the residual norm, the 8-bit values and the clipping against other definitions: torch in
64 bits, torch's own e4m3 conversion, finite differences, brute force."""
import math

import numpy as np
import pytest
import torch

from oracle import layer as ol


def rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("D", [1, 7, 128, 300])
def test_rmsnorm_against_torch(D):
    h, w = rng(0).standard_normal((5, D)), rng(1).standard_normal(D)
    want = torch.nn.functional.rms_norm(torch.tensor(h), (D,), torch.tensor(w), 1e-5).numpy()
    assert np.abs(ol.rmsnorm(h, w, 1e-5) - want).max() < 1e-13


@pytest.mark.parametrize("with_dh", [False, True])
def test_rmsnorm_gradients_against_differences(with_dh):
    r, eps, step = rng(2), 0.3, 1e-6
    h, w, dout, dh = (r.standard_normal(s) for s in ((3, 20), (20,), (3, 20), (3, 20)))
    dh = dh if with_dh else None
    f = lambda h, w: np.sum(ol.rmsnorm(h, w, eps) * dout) + (0 if dh is None else np.sum(h * dh))  # noqa: E731
    d, dw, size, wsize = ol.rmsnorm_backward(h, w, dout, dh, eps)
    for got, which, at in ((d, 0, h), (dw, 1, w)):
        v = r.standard_normal(at.shape)
        a = [h, w]
        a[which] = at + step * v
        up = f(*a)
        a[which] = at - step * v
        assert abs((up - f(*a)) / (2 * step) - np.sum(got * v)) < 1e-7
    assert (size >= np.abs(d)).all() and (wsize >= np.abs(dw) - 1e-15).all()


def test_e4m3_against_torch():
    v = np.concatenate([np.linspace(-448, 448, 4001), np.exp2(rng(3).uniform(-14, 8, 4000)), [0.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    v = v.astype(np.float32).astype(np.float64)
    assert np.array_equal(ol.e4m3(v), torch.tensor(v, dtype=torch.float32).to(torch.float8_e4m3fn).double().numpy())
    assert np.all(np.abs(ol.e4m3(v) - v) <= 2.0 ** -4 * np.abs(v) + 2.0 ** -10)


def test_scales():
    for amax in (448.0, 448.0000001, 447.0, 1.75, 1.7500001, 1.0, 3.4e38, 1e-30):
        s = ol.scale_of(amax)
        assert math.log2(s) == round(math.log2(s)) and amax / s <= 448 < 2 * amax / s
    assert ol.scale_of(0.0) == ol.scale_of(1e-45) == 2.0 ** -126
    assert math.isnan(ol.scale_of(math.inf)) and math.isnan(ol.scale_of(math.nan))


def test_product_of_values_that_need_no_rounding():
    r = rng(4)
    x, w = r.integers(-8, 9, (4, 300)) * 1.0, r.integers(-8, 9, (200, 300)) * 2.0 ** -4
    out, size = ol.linear(*ol.quantise(x), *ol.quantise_weight(w))
    assert np.array_equal(out, x @ w.T) and (size >= np.abs(out)).all()


@pytest.mark.parametrize("most", [0.5, 100.0])
def test_clip_against_torch(most):
    g = [rng(5).standard_normal(s) for s in ((3, 4), (7,), (1,))]
    t = [torch.tensor(x, requires_grad=True) for x in g]
    for x, y in zip(t, g):
        x.grad = torch.tensor(y)
    norm = torch.nn.utils.clip_grad_norm_(t, most)
    n, out = ol.clip(g, most)
    assert abs(n - float(norm)) < 1e-12
    for x, y in zip(out, t):
        assert np.abs(x - y.grad.numpy()).max() < 2e-6  # torch divides by norm + 1e-6


def test_mistakes_are_seen():
    """Planted mistakes in copies of the formulas fail against the oracle."""
    r = rng(6)
    h, w, dout = r.standard_normal((4, 64)), r.standard_normal(64), r.standard_normal((4, 64))
    d, dw, _, _ = ol.rmsnorm_backward(h, w, dout, None, 1e-5)
    inv = 1 / np.sqrt(np.mean(h * h, -1, keepdims=True) + 1e-5)
    g = dout * w
    assert np.abs(inv * g - d).max() > 1e-2                                                       # no shared term
    assert np.abs(inv * g - h * inv ** 2 * np.mean(g * h, -1, keepdims=True) - d).max() > 1e-3  # a power too few
    assert np.abs((dout * h).sum(0) - dw).max() > 1e-2                                            # dw not normalised
    assert ol.scale_of(460.0) != ol.scale_of(440.0)                                               # 448, not 512
