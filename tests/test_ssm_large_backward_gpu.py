"""Backward passes over tensors of more than 2^31 values, against calls on their two parts.

Gradients of tokens are the same arithmetic in both (conv, norm: the same bits) or differ by the float32
roundings of states found in other pieces (scan).  Sums over all tokens are float32 in another order: n
additions in a row lose at most n 2^-24 of the terms' magnitudes, and n is below 512 here (128 tokens a
thread or two rows a team in turn, then rows of partial sums in 32 slices): 2^-15 of them.
"""
import pytest
import torch

import matrix_state_nonlinear_gb300 as pkg
from test_ssm_gpu import BF16, DEV, built, rand, scan_case  # noqa: F401

pytestmark = pytest.mark.gpu
T, C = 1_100_000, 2048
CUT = (T - 12_000) // 128 * 128


def test_conv_backward():
    x, dout = (torch.randn(1, T, C, device=DEV, dtype=BF16) for _ in range(2))
    w, b = rand((C, 4), 1, 0.6, torch.float32), rand((C,), 2, 0.3, torch.float32)
    g = pkg.conv_silu_backward(x, w, b, dout)
    first = pkg.conv_silu_backward(x[:, :CUT].contiguous(), w, b, dout[:, :CUT].contiguous())
    last = pkg.conv_silu_backward(x[:, CUT:].contiguous(), w, b, dout[:, CUT:].contiguous(), x[:, CUT - 3:CUT].contiguous())
    assert torch.equal(g["dx"][:, :CUT - 3], first["dx"][:, :CUT - 3]) and torch.equal(g["dx"][:, CUT:], last["dx"])
    size = 1.1 * dout.abs().sum((0, 1), dtype=torch.float32)
    assert bool(((g["dbias"] - first["dbias"] - last["dbias"]).abs() <= 2.0 ** -15 * size).all())
    size = 1.1 * torch.linalg.vector_norm(x[0], dim=0, dtype=torch.float32) * torch.linalg.vector_norm(dout[0], dim=0, dtype=torch.float32)
    assert bool(((g["dw"] - first["dw"] - last["dw"]).abs() <= 2.0 ** -15 * size[:, None]).all())


def test_norm_backward():
    y, gate, dout = (torch.randn(T, C, device=DEV, dtype=BF16) for _ in range(3))
    w, b = 1.0 + rand((C,), 2, 0.2, torch.float32), rand((C,), 3, 0.2, torch.float32)
    g = pkg.gate_groupnorm_backward(y, gate, w, b, dout, 32)
    first = pkg.gate_groupnorm_backward(y[:CUT], gate[:CUT], w, b, dout[:CUT], 32)
    last = pkg.gate_groupnorm_backward(y[CUT:], gate[CUT:], w, b, dout[CUT:], 32)
    for n in ("dy", "dg_pre"):
        assert torch.equal(g[n][:CUT], first[n]) and torch.equal(g[n][CUT:], last[n]), n
    # a team adds T / slots rows in turn, about 7300, then 152 slots or so in slices: 2^13 2^-24 at most;
    # the terms dp n and dp by their norms (|dp| <= 1.1 |dout| (|gate| + 1), n of unit variance)
    size = 1.1 * torch.linalg.vector_norm(dout, dim=0, dtype=torch.float32) * \
        (torch.linalg.vector_norm(gate, dim=0, dtype=torch.float32) + T ** 0.5)
    for n in ("dw", "dbias"):
        assert bool(((g[n] - first[n] - last[n]).abs() <= 2.0 ** -11 * size).all()), n


def test_scan_backward():
    N, K, V = 32, 64, 64
    s = scan_case(1, T, N, 1, K, 1, seed=140, h0=False)
    s.update(v=torch.randn(1, T, N, V, device=DEV, dtype=BF16), w_r=rand((N, V), 141, 1.0, torch.float32))
    dy = torch.randn(1, T, N, V, device=DEV, dtype=BF16)
    cut = lambda lo, hi: {n: t[:, lo:hi] if n in ("q", "k", "v", "a") else t for n, t in s.items()}  # noqa: E731
    Hs = pkg.ssm_forward_train(s)[2]
    g = pkg.ssm_backward(s, Hs, dy)
    del Hs
    front = cut(0, CUT)
    _, H, Hs = pkg.ssm_forward_train(front)
    back = dict(cut(CUT, T), H0=H)
    last = pkg.ssm_backward(back, pkg.ssm_forward_train(back)[2], dy[:, CUT:].contiguous())
    first = pkg.ssm_backward(front, Hs, dy[:, :CUT].contiguous(), last["dH0"])
    for n in ("dq", "dk", "dv", "da"):
        for part, want in ((g[n][:, CUT:], last[n]), (g[n][:, :20_000], first[n][:, :20_000]),
                           (g[n][:, CUT - 20_000:CUT], first[n][:, CUT - 20_000:])):
            off = float((part.float() - want.float()).abs().max())
            assert off <= 2.0 ** -7 * float(want.float().abs().max()), (n, off)
    assert float((g["dH0"] - first["dH0"]).abs().max()) <= 2.0 ** -14 * float(first["dH0"].abs().max())
    size = torch.linalg.vector_norm(dy[0], dim=0, dtype=torch.float32) * torch.linalg.vector_norm(s["v"][0], dim=0, dtype=torch.float32)
    assert bool(((g["dw_r"] - first["dw_r"] - last["dw_r"]).abs() <= 2.0 ** -14 * size).all())
    for n in ("dalpha", "dbeta"):  # 2^-14 of the terms' magnitudes: of da, and of d g, which are of da's size
        assert bool(((g[n] - first[n] - last[n]).abs() <= 2.0 ** -14 * g["da"].float().abs().sum((0, 1)).clamp(min=1)).all()), n
    assert pkg.stream_status() == 0
