"""Rows and weights of 2^31 - 1 values, the longest that the calls take, in 8 bits: their ends are those of the same
values alone."""
import pytest
import torch

import matrix_state_nonlinear_gb300 as pkg
from test_layer_gpu import BF16, DEV, built  # noqa: F401
from test_layer_large_gpu import room  # noqa: F401

pytestmark = pytest.mark.gpu
TOP = 2 ** 31 - 1
END = TOP % 128 + 128 * 7  # from a block's start on


def values(n):
    """Some values over and over."""
    some = torch.randn(1_000_003, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(BF16)
    t = torch.empty(n, dtype=BF16, device=DEV)
    for i in range(0, n, len(some)):
        t[i:i + len(some)] = some[:min(len(some), n - i)]
    return t


def ends_as(q, s, a, b):
    """The last values and scales of (q, s), one row, are those of (a, b)."""
    bits = lambda t: t.view(torch.uint8).flatten()  # noqa: E731
    return torch.equal(bits(q.flatten()[-a.numel():]), bits(a)) and torch.equal(bits(s)[-b.numel():], bits(b))


def test_a_row():
    x = values(TOP)
    q, s = pkg.quantise_fp8(x)
    assert s.shape == (2 ** 24,) and ends_as(q, s, *pkg.quantise_fp8(x[-END:].clone()))


def test_a_weight_of_one_channel():
    w = values(TOP).view(1, TOP)
    q, s = pkg.quantise_weight_fp8(w)
    assert s.shape == (1, 2 ** 24) and ends_as(q, s, *pkg.quantise_weight_fp8(w[:, -END:].clone()))


def test_a_weight_of_one_value_a_channel():
    w = values(TOP).view(TOP, 1)
    q, s = pkg.quantise_weight_fp8(w)
    a, b = pkg.quantise_weight_fp8(w[-END:].clone())
    assert s.shape == (2 ** 24, 1) and torch.equal(q[-END:].view(torch.uint8), a.view(torch.uint8))
    assert torch.equal(s[-8:].view(torch.uint8), b.view(torch.uint8))
