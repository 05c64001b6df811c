"""The gradients' norm and clipping at the ends of float32's range.  Tolerances as in the clip's own tests."""
import numpy as np
import pytest
import torch

import matrix_state_nonlinear_gb300 as pkg
from test_layer_gpu import BF16, DEV, F32, built, check_clip, tensors  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bit", [0, 7, 15, 16, 22])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_values_of_one_bit(bit, sign):
    """float32 values below 2^-126 with any one bit of theirs: no bit is a sign but the highest."""
    value = sign * 2.0 ** (bit - 149)
    for n in (1, 1000, 40003):
        grads = [torch.full((n,), value, dtype=F32, device=DEV), torch.zeros(50, device=DEV)]
        out = [torch.empty_like(g) for g in grads]
        assert float(grads[0][0]) == value
        most = 2.0 ** -149
        check_clip(grads, most, out, pkg.clip_grad_norm(grads, most, out=out))
        assert torch.equal(pkg.grad_norm(grads), pkg.clip_grad_norm(grads, 1.0))


@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("most", [1e-3, 1e-12, 1e-30])
@pytest.mark.parametrize("off", [0, 1])
def test_factors_below_the_range(kind, most, off):
    """max_norm / norm below 2^-126, where the clipped values are ordinary numbers; in whole accesses and beside them."""
    most = float(np.float32(most))
    grads = tensors([9000, 37, 50001], 80, [kind] * 3, 1e37)
    grads[0][5] = 3e38
    grads = [g[off:] for g in grads]
    before = [g.clone() for g in grads]
    out = [torch.empty_like(g) for g in grads]
    norm = pkg.clip_grad_norm(grads, most, out=out)
    assert most / 1e40 < 2.0 ** -126
    check_clip(before, most, out, norm)
    pkg.clip_grad_norm(grads, most)
    assert all(torch.equal(a, b) for a, b in zip(grads, out))
