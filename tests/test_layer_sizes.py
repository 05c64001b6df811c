"""Sizes at the edges of the layer's calls: rows that do not fit 32 bits or barely do, no rows at all.

No GPU is used: stand-ins for tensors, and a library that says that it was reached."""
import pytest
import torch

import __graft_entry__
import matrix_state_nonlinear_gb300 as pkg
from matrix_state_nonlinear_gb300 import m2rnn as binding
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


def test_no_tokens_in_8_bits(stub):  # noqa: F811
    """8-bit rows of any width where there are none: their strides say nothing."""
    w, sw = t(128, 1008, dtype=FP8), t(1, 8, dtype=E8M0)
    for x, s in (((0, 1000), (0, 8)), ((3, 0, 1000), (3, 0, 8))):
        w.shape, w.is_contiguous, w.stride = torch.Size((128, 1000)), lambda: False, lambda: (1008, 1)
        with pytest.raises(Reached):
            pkg.linear_fp8(t(*x, dtype=FP8), t(*s, dtype=E8M0), w, sw, out=t(*x[:-1], 128))
    with pytest.raises(Reached):
        pkg.quantise_fp8(t(0, 1000), out=t(0, 1000, dtype=FP8), scales=t(0, 8, dtype=E8M0))
    with pytest.raises(Reached):
        pkg.add_rmsnorm_fp8(t(0, 1000), None, t(1000, dtype=F32), out=t(0, 1000, dtype=FP8), scales=t(0, 8, dtype=E8M0))


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return binding.load_library()


@pytest.mark.parametrize("n", [2 ** 31 - 129, 2 ** 31 - 128, 2 ** 31 - 127, 2 ** 31 - 1])
def test_blocks_of_the_longest_rows_are_counted_right(lib, n):
    """Sizes next to 2^31, whose blocks are counted by adding 127."""
    blocks = -(-n // 128)
    assert lib.m2rnn_linear_quantise_workspace_bytes(1, 1, n) == 128 * blocks + blocks
    assert lib.m2rnn_quantise_fp8(None, 0, n, None, 1 << 31, None, 0, n, None) == binding.OK
    # as many rows as their blocks allow and one more: refused before any address is looked at
    most = 0x7ffffff0 * 16 // blocks
    assert lib.m2rnn_quantise_fp8(None, 0, n, None, 1 << 31, None, most, n, None) == binding.ERR_UNSUPPORTED
    assert lib.m2rnn_quantise_fp8(None, 0, n, None, 1 << 31, None, most - 1, n, None) == binding.ERR_INVALID_ARG
    # 2^24 blocks of weights by 127 are fewer than 2^31, by 128 they are not
    for N, K in ((n, 127 * 128), (127 * 128, n)):
        assert lib.m2rnn_quantise_weight_fp8(None, 0, K, None, 1 << 31, None, N, K, None) == binding.ERR_INVALID_ARG
    for N, K in ((n, 128 * 128 + 1), (128 * 128 + 1, n)):
        assert lib.m2rnn_quantise_weight_fp8(None, 0, K, None, 1 << 31, None, N, K, None) == binding.ERR_UNSUPPORTED
