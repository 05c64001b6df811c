"""The scan under strong decay: many tokens of one chunk that forget the state, alone and followed by
slow ones, so that the sum of log f over a chunk runs into the thousands while the weights between
neighbouring tokens stay of ordinary size.

Every result of both directions is held to the tolerances of test_ssm_gpu.py.  They do not widen with
the decay: a weight exp(c_t - c_s) d_s depends on the tokens from s to t alone, so the size of the sums
before s must not enter its error.  With positive q, k, v, dy no terms cancel: the bounds are then
relative to the results themselves, and the error of single weights shows.
"""
import numpy as np
import pytest
import torch

import matrix_state_nonlinear_gb300 as pkg
from oracle import ssm_block as ob
from test_ssm_gpu import BF16, DEV, built, check_forward, f64, oracle_inputs, rand, scan_case, within  # noqa: F401

pytestmark = pytest.mark.gpu


def check_backward(s, dy, dH=None):
    want = ob.ssm_backward(**oracle_inputs(s), dy=f64(dy), dH_T=f64(dH))
    size = ob.ssm_backward(**oracle_inputs(s, True), dy=np.abs(f64(dy)), dH_T=None if dH is None else np.abs(f64(dH)),
                           bound=True)
    g = pkg.ssm_backward(s, pkg.ssm_forward_train(s)[2], dy, dH)
    for n in ("dq", "dk", "dv"):
        within(g[n], want[n], 2.0 ** -8 * (np.abs(want[n]) + size[n]) + 1e-6, n)
    within(g["da"], want["da"], 2.0 ** -8 * np.abs(want["da"]) + 2.0 ** -10 * size["da"].max() + 1e-6, "da")
    for n in ("dalpha", "dbeta", "dw_r", "dH0"):
        within(g[n], want[n], 2.0 ** -14 * size[n] + 1e-6, n)


def case(kind, T, N, G, K, V, seed, positive, h0):
    """Tokens with the decays of ``kind``; resetting tokens (d = 200) write nothing themselves."""
    s = scan_case(1, T, N, G, K, V, seed=seed, h0=h0)
    s["a"], s["alpha"] = decays(kind, T, N)
    s["beta"] = torch.zeros_like(s["beta"])
    s["k"] = torch.where((s["a"] > 100).any(-1)[..., None, None], torch.zeros_like(s["k"]), s["k"])
    if positive:
        s.update({n: s[n].abs() for n in ("q", "k", "v")})
    return s


def decays(kind, T, N):
    """Logits [1, T, N] and alpha [N] of one kind of sequence."""
    a = rand((1, T, N), 201, 1.0, torch.float32)
    alpha = torch.full((N,), 1.0, device=DEV)
    if kind == "large steps":        # d near 40, f = exp(-80)
        a, alpha = 40.0 + 2.0 * a, 2.0 * alpha
    elif kind == "steady heads":     # d near 1.3, alpha = 4: 32 tokens decay by about 2^-245
        a, alpha = 1.0 + 0.05 * a, 4.0 * alpha
    elif kind == "fast heads":       # d near 5, alpha = 16
        a, alpha = 5.0 + a, 16.0 * alpha
    elif kind == "resets then slow":  # three quarters of a chunk forget everything
        a = torch.where((torch.arange(T, device=DEV) % 128 < 96)[None, :, None], torch.full_like(a, 200.0), a - 2.0)
    else:                            # a reset every eighth token, slow ones between
        a = torch.where((torch.arange(T, device=DEV) % 8 == 0)[None, :, None], torch.full_like(a, 200.0), a - 1.0)
    return a.to(BF16), alpha


KINDS = ["steady heads", "large steps", "fast heads", "resets then slow", "resets between"]


@pytest.mark.parametrize("K,V", [(64, 64), (128, 64), (40, 24)])
@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("kind", KINDS)
def test_every_result(kind, positive, K, V):
    s = case(kind, 300, 4, 2, K, V, 210, positive, True)
    check_forward(s, *pkg.ssm_forward(s))
    dy = rand((1, 300, 4, V), 211)
    check_backward(s, dy.abs() if positive else dy, rand((1, 4, K, V), 212, 0.5, torch.float32))
    assert pkg.stream_status() == 0


@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("kind", KINDS)
def test_one_readout(kind, positive):
    """Only the last token of a chunk is read: each sum of the gate's gradient has few terms.  Sixteen
    heads, each with sums of its own."""
    s = case(kind, 128, 16, 16, 64, 64, 220, positive, False)
    dy = torch.zeros(1, 128, 16, 64, dtype=BF16, device=DEV)
    dy[:, -1] = rand((1, 16, 64), 221)
    check_backward(s, dy.abs() if positive else dy)


def test_decays_between_chunks_backward():
    """Decays of one token from none to complete (f from 1 to 0), over chunks and pieces, backwards."""
    s = scan_case(1, 1500, 2, 1, 64, 64, seed=101)
    s["a"] = rand((1, 1500, 2), 102, 12.0, torch.float32).to(BF16)
    check_backward(s, rand((1, 1500, 2, 64), 103))


def test_inert_and_resetting_tokens_gate_gradients():
    """Inert and resetting tokens among ordinary ones: the gate's gradients too."""
    s = scan_case(1, 150, 2, 1, 64, 64, seed=70)
    s["a"][:, 20:40] = -float("inf")
    s["a"][:, 64] = s["a"][:, 100] = 200.0
    s["k"][:, 64] = s["k"][:, 100] = 0
    check_backward(s, rand((1, 150, 2, 64), 71))


@pytest.mark.parametrize("shape", [(2, 128, 8, 1, 128, 24), (1, 85, 16, 16, 64, 64), (1, 400, 6, 2, 40, 72)])
@pytest.mark.parametrize("alpha", [0.5, 1.0, 2.0])
def test_large_steps_among_small_ones(shape, alpha):
    """d from 0 to 35, so that what a chunk's slow tokens leave in a sum would count many times over at its
    fast ones, whose own gradient of log f is next to nothing.  dalpha weighs that gradient by d."""
    B, T, N, _, _, V = shape
    s = scan_case(*shape, seed=230, h0=False)
    s.update({n: s[n].abs() for n in ("q", "k", "v")})
    s["a"] = (10.0 + 8.0 * rand((B, T, N), 231, 1.0, torch.float32)).to(BF16)
    s["alpha"], s["beta"] = torch.full_like(s["alpha"], alpha), torch.zeros_like(s["beta"])
    check_forward(s, *pkg.ssm_forward(s))
    check_backward(s, rand((B, T, N, V), 232))
    check_backward(s, rand((B, T, N, V), 233).abs())
