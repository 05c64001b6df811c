"""The norm's last rows in tensors of more than 2^31 values against the 64-bit definition, whatever a smaller call of
the same kernels gives.  Seeded throughout; tolerances as in the norm's own tests."""
import pytest
import torch

import matrix_state_nonlinear_gb300 as pkg
from oracle import layer as ol
from test_layer_gpu import BF16, DEV, F32, built, check_h, check_quantised, f64, rand, within  # noqa: F401
from test_layer_large_gpu import OVER, fill, room  # noqa: F401

pytestmark = pytest.mark.gpu
LAST = 50


@pytest.mark.parametrize("D", [2048, 2049])
@pytest.mark.parametrize("odd", [0, 1])
def test_norm(D, odd):
    """odd: x one value behind a 16-byte boundary, so that rows are read value by value."""
    rows = OVER // D + 777
    flat = torch.empty(rows * D + odd, dtype=BF16, device=DEV)
    x, r, w = flat[odd:].view(rows, D), fill((rows, D), 2), 1 + rand((D,), 3, 0.2, F32)
    x.copy_(fill((rows, D), 1))
    out, h = pkg.add_rmsnorm(x, r, w, 1e-5)
    last = lambda t: t[-LAST:]  # noqa: E731
    check_h(last(h), last(x), last(r))
    want = ol.rmsnorm(f64(last(h)), f64(w), 1e-5)
    within(last(out), want, (2.0 ** -8 + 2.0 ** -17) * abs(want))
    del out
    q, s, h = pkg.add_rmsnorm_fp8(x, r, w, 1e-5, h=h)
    check_quantised(last(q), last(s), want)
    del q, s
    g = pkg.add_rmsnorm_backward(h, w, x, r, 1e-5)
    d, _, size, _ = ol.rmsnorm_backward(f64(last(h)), f64(w), f64(last(x)), f64(last(r)), 1e-5)
    within(last(g["dx"]), d, 2.0 ** -8 * abs(d) + 2.0 ** -16 * size)
