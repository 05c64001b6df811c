"""Sizes at the edges of the layer's calls: rows that do not fit 32 bits, no rows at all.

No GPU is used: stand-ins for tensors, and a library that says that it was reached."""
import pytest
import torch

import matrix_state_nonlinear_gb300 as pkg
from test_layer_binding import BF16, E8M0, F32, FP8, Reached, stub  # noqa: F401
from test_ssm_binding import Fake

WIDE = 2 ** 32 + 16  # 16, cut down to 32 bits


def t(*shape, dtype=BF16):
    return Fake(0, *shape, dtype=dtype)


ROWS = {
    "add_rmsnorm": lambda D: pkg.add_rmsnorm(t(2, D), t(2, D), t(D, dtype=F32), out=t(2, D), h=t(2, D)),
    "add_rmsnorm_fp8": lambda D: pkg.add_rmsnorm_fp8(t(2, D), None, t(D, dtype=F32), out=t(2, D, dtype=FP8),
                                                     scales=t(2, (D + 127) // 128, dtype=E8M0)),
    "add_rmsnorm_backward": lambda D: pkg.add_rmsnorm_backward(t(2, D), t(D, dtype=F32), t(2, D), grads=dict(dx=t(2, D), dw=t(D, dtype=F32)),
                                                               workspace=t(4096, dtype=torch.uint8)),
}


@pytest.mark.parametrize("name", sorted(ROWS))
def test_rows_that_do_not_fit_32_bits_are_refused(stub, name):  # noqa: F811
    with pytest.raises(Reached):
        ROWS[name](16)
    with pytest.raises(ValueError, match="2\\^31"):
        ROWS[name](WIDE)
