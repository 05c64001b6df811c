"""Taps at any float32 address: a weight that is a view into a flat buffer of parameters."""
import pytest
import torch

import matrix_state_nonlinear_gb300 as pkg
from test_ssm_gpu import built, conv_case, rand  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("offset", [1, 2, 3, 4])
@pytest.mark.parametrize("shape", [(2, 70, 24), (1, 1, 1024), (2, 65, 7), (3, 4099, 64)])
def test_taps_of_a_flat_buffer(shape, offset):
    """The same bits, forward, single token and backward, wherever the taps lie."""
    x, w, bias, window = conv_case(*shape, seed=300)
    flat = torch.full((offset + w.numel() + 3,), float("nan"), device=w.device)
    view = flat[offset:offset + w.numel()].view_as(w)
    view.copy_(w)
    for a, b in zip(pkg.conv_silu_window(x, view, bias, window), pkg.conv_silu_window(x, w, bias, window)):
        assert torch.equal(a, b)
    token, win = x[:, 0].contiguous(), window.clone()
    assert torch.equal(pkg.conv_silu_step(token, view, bias, win)[0], pkg.conv_silu_step(token, w, bias, window.clone())[0])
    dout = rand(shape, 301)
    got, want = pkg.conv_silu_backward(x, view, bias, dout, window), pkg.conv_silu_backward(x, w, bias, dout, window)
    assert all(torch.equal(got[n], want[n]) for n in want)
