"""Sizes at the edge of 32-bit counts: refused or counted right, before anything is launched.

No GPU is used: the entries return on their size checks, the byte counts are host arithmetic.  Pointers
are stand-ins that nothing reads.
"""
import pytest
import torch

import __graft_entry__
from matrix_state_nonlinear_gb300 import m2rnn as binding
from matrix_state_nonlinear_gb300 import ssm
from test_ssm_binding import Fake, library  # noqa: F401
import matrix_state_nonlinear_gb300 as pkg

TOP, TOKENS = 2 ** 31 - 1, 2 ** 31 - 128
P = 1 << 20


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return binding.load_library()


@pytest.mark.parametrize("T", [TOKENS + 1, TOP])
def test_sequences_too_long_are_refused(lib, T):
    n = binding.ERR_UNSUPPORTED
    assert lib.m2rnn_conv_silu_window_bf16(P, P, P, P, P, P, 1, T, 1, T, 1, None) == n
    assert lib.m2rnn_conv_silu_backward_bf16(*[P] * 9, 1, T, 1, T, 1, P, 1 << 62, None) == n
    assert lib.m2rnn_ssm_forward_bf16(*[P] * 11, None, 1, T, 1, 1, 1, 1, P, 1 << 62, None) == n
    assert lib.m2rnn_ssm_backward_bf16(*[P] * 18, None, 1, T, 1, 1, 1, 1, P, 1 << 62, None) == n
    assert lib.m2rnn_ssm_states_bytes(1, T, 1, 1, 1) == 0
    assert lib.m2rnn_ssm_workspace_bytes(1, T, 1, 1, 1, 1, 1) == 0
    assert lib.m2rnn_conv_silu_backward_workspace_bytes(1, T, 1) == 0


def test_the_longest_sequences_are_counted_right(lib):
    chunks = (TOKENS + 127) // 128
    assert lib.m2rnn_ssm_states_bytes(1, TOKENS, 1, 1, 1) == 4 * (chunks + 1)
    assert lib.m2rnn_conv_silu_backward_workspace_bytes(1, TOKENS, 8) > 0


def test_counts_of_sums_too_large_are_refused(lib):
    n = binding.ERR_UNSUPPORTED
    C = (2 ** 31 - 32) // 5
    assert lib.m2rnn_conv_silu_backward_workspace_bytes(1, 1, C) == 4 * 5 * C
    assert lib.m2rnn_conv_silu_backward_workspace_bytes(1, 1, C + 1) == 0
    assert lib.m2rnn_conv_silu_backward_bf16(*[P] * 9, 1, 1, C + 1, C, C, P, 1 << 62, None) == n
    B = 2 ** 28  # of 16 stretches of eight tokens each: 2^32 rows of partial sums
    assert lib.m2rnn_conv_silu_backward_bf16(*[P] * 9, B, 128, 1, 128, 1, P, 1 << 62, None) == n
    assert lib.m2rnn_conv_silu_backward_workspace_bytes(B, 128, 1) == 0
    N = (2 ** 31 - 32) // 130
    assert lib.m2rnn_ssm_workspace_bytes(1, 1, N, 1, 1, 128, 1) > 0
    assert lib.m2rnn_ssm_workspace_bytes(1, 1, N + 1, 1, 1, 128, 1) == 0
    assert lib.m2rnn_ssm_backward_bf16(*[P] * 18, None, 1, 1, N + 1, 1, 1, 128, P, 1 << 62, None) == n
    D = 2 ** 30 - 16
    assert lib.m2rnn_gate_groupnorm_backward_workspace_bytes(1, D, D // 16) > 0
    assert lib.m2rnn_gate_groupnorm_backward_workspace_bytes(1, D + 16, D // 16 + 1) == 0
    assert lib.m2rnn_gate_groupnorm_backward(P, 0, P, P, P, 1e-5, P, P, P, P, P, 1, D + 16, D // 16 + 1, P, 1 << 62, None) == n


def test_the_binding_refuses_sizes_that_do_not_fit(library):  # noqa: F811
    """ctypes would pass 2^32 + 1 tokens on as one."""
    big, f32 = 2 ** 32 + 1, torch.float32
    w, b = Fake(0, 1, 4, dtype=f32), Fake(0, 1, dtype=f32)
    one = lambda *s, dtype=torch.bfloat16: Fake(0, *s, dtype=dtype)  # noqa: E731
    x = one(1, big, 1)
    s = dict(q=one(1, big, 1, 1), k=one(1, big, 1, 1), v=one(1, big, 1, 1), a=one(1, big, 1), alpha=b, beta=b, w_r=one(1, 1, dtype=f32))
    y = one(1, big)
    for call in (lambda: pkg.conv_silu_window(x, w, b, out=x, window_out=one(1, 3, 1)),
                 lambda: pkg.conv_silu_step(one(big, 1), w, b, one(big, 3, 1), out=one(big, 1)),
                 lambda: pkg.conv_silu_backward(x, w, b, x, workspace=x),
                 lambda: pkg.ssm_forward(s, y=s["v"], workspace=x),
                 lambda: pkg.ssm_backward(s, one(64, dtype=torch.uint8), s["v"], workspace=x),
                 lambda: pkg.ssm_step(one(big, 1, 1), one(big, 1, 1), one(big, 1, 1), one(big, 1), b, b, s["w_r"],
                                      one(big, 1, 1, 1, dtype=f32), y=one(big, 1, 1)),
                 lambda: pkg.gate_groupnorm(y, None, one(big, dtype=f32), None, big, out=y),
                 lambda: pkg.gate_groupnorm_backward(y, None, one(big, dtype=f32), None, y, big, workspace=x),
                 lambda: ssm.ssm_states_bytes(1, big, 1, 1, 1), lambda: ssm.ssm_workspace_bytes(1, big, 1, 1, 1, 1)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
