"""The selective state space block on the GPU against the fp64 oracle.

Tolerances, derived from the arithmetic:
 * bf16 results of fp32 arithmetic (conv, norm, single token): half a bf16 ulp (2^-9 of the
   value) plus fp32 rounding, held to 2^-8 |want| + 1e-5.
 * The scan's y, dq, dk, dv: the tensor-core operands that are not inputs (decayed scores,
   states, state gradients) are rounded to bf16, an error of at most 2^-9 of each term, two such
   roundings per term at most, and one on the result: 2^-8 (|want| + A), A the sum of the terms'
   magnitudes (the oracle on absolute inputs).
 * float32 results (states, dH0, parameter gradients): states are carried in float32 and enter
   products as two bf16 values (2^-17 of each term), gates are float32 sums over at most 128
   tokens: 2^-14 A.  da: the same before its own rounding, with sums over a chunk's tokens:
   2^-8 |want| + 2^-10 max A.
"""
import numpy as np
import pytest
import torch

import __graft_entry__
import matrix_state_nonlinear_gb300 as pkg
from matrix_state_nonlinear_gb300 import m2rnn as binding
from oracle import ssm_block as ob

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    __graft_entry__.build()
    pkg.load_library()


def rand(shape, seed, scale=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(DEV)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def within(got, want, tol, what=""):
    over = np.abs(f64(got) - want) - tol
    assert np.isfinite(f64(got)).all() and float(over.max(initial=-1.0)) <= 0.0, (what, float(over.max()))


# ---------------------------------------------------------------- convolution
CONV = [(1, 1, 8), (2, 2, 16), (3, 3, 24), (2, 70, 24), (1, 129, 1024), (2, 65, 7), (1, 5, 1), (2, 200, 40)]


def conv_case(B, T, C, seed=0, pad=0):
    x = rand((B, T, C + pad), seed, 1.5)[:, :, :C]
    w, bias = rand((C, 4), seed + 1, 0.6, torch.float32), rand((C,), seed + 2, 0.3, torch.float32)
    return x, w, bias, rand((B, 3, C), seed + 3, 1.5)


@pytest.mark.parametrize("shape", CONV)
@pytest.mark.parametrize("with_window,with_bias,pad", [(True, True, 8), (False, False, 0), (True, False, 3)])
def test_conv_window(shape, with_window, with_bias, pad):
    x, w, bias, window = conv_case(*shape, pad=pad)
    bias, window = bias if with_bias else None, window if with_window else None
    out, after = pkg.conv_silu_window(x, w, bias, window)
    want, wafter, _, _ = ob.conv_window(f64(x), f64(w), f64(bias), f64(window))
    within(out, want, 2.0 ** -8 * np.abs(want) + 1e-5)
    assert np.array_equal(f64(after), wafter)


@pytest.mark.parametrize("C", [8, 40, 13])
def test_conv_tokens_continue_a_prompt(C):
    """A prompt cut in two calls and then single tokens, windows in place: the bits of one call."""
    x, w, bias, window = conv_case(2, 90, C, seed=5)
    whole, after = pkg.conv_silu_window(x, w, bias, window)
    win = window.clone()
    parts = [pkg.conv_silu_window(x[:, :70], w, bias, win, window_out=win)[0]]
    for t in range(70, 90):
        parts.append(pkg.conv_silu_step(x[:, t], w, bias, win)[0].unsqueeze(1))
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(win, after)
    empty, same = pkg.conv_silu_window(x[:, :0], w, bias, window)
    assert empty.shape == (2, 0, C) and torch.equal(same, window)


@pytest.mark.parametrize("shape", CONV)
@pytest.mark.parametrize("with_window,pad", [(True, 8), (False, 1)])
def test_conv_backward(shape, with_window, pad):
    x, w, bias, window = conv_case(*shape, seed=7, pad=pad)
    window = window if with_window else None
    dout = rand(shape, 11)
    g = pkg.conv_silu_backward(x, w, bias, dout, window)
    want = ob.conv_window_backward(f64(x), f64(w), f64(bias), f64(dout), f64(window))
    for n in ("dx", "dwindow"):
        within(g[n], want[n], 2.0 ** -8 * np.abs(want[n]) + 1e-5, n)
    # float32 sums of B T terms, each a few 2^-22 off its magnitude (|dout| <= 1.1 |slope| bound)
    X = np.abs(ob.conv_window(f64(x), f64(w), f64(bias), f64(window))[3])
    terms = 1.1 * np.abs(f64(dout))
    within(g["dbias"], want["dbias"], 2.0 ** -18 * terms.sum((0, 1)) + 1e-7, "dbias")
    for j in range(4):
        bound = (terms * X[:, j:j + shape[1]]).sum((0, 1))
        within(g["dw"][:, j], want["dw"][:, j], 2.0 ** -18 * bound + 1e-7, "dw")


# ---------------------------------------------------------------- selective scan
# B, T, N, Nqk, K, V: one token, chunk edges, odd widths, both widest, shared and grouped heads,
# long enough to be cut into segments.
SCAN = [(1, 1, 1, 1, 16, 16), (2, 63, 2, 1, 64, 64), (1, 64, 2, 2, 64, 64), (1, 65, 2, 1, 32, 64),
        (2, 130, 4, 2, 40, 24), (1, 200, 2, 2, 128, 128), (1, 77, 3, 3, 8, 8), (1, 300, 2, 1, 64, 128),
        (1, 129, 2, 1, 128, 64), (1, 100, 1, 1, 1, 1), (1, 90, 2, 2, 17, 33), (1, 150, 2, 1, 112, 80),
        (1, 3000, 1, 1, 64, 64), (1, 2100, 2, 1, 128, 128), (5, 70, 33, 11, 16, 48)]


def scan_case(B, T, N, G, K, V, seed=0, h0=True, fused=False):
    s = dict(alpha=torch.exp(rand((N,), seed, 0.8, torch.float32)), beta=rand((N,), seed + 1, 1.0, torch.float32),
             w_r=rand((N, V), seed + 2, 1.0, torch.float32), H0=rand((B, N, K, V), seed + 3, 0.4, torch.float32) if h0 else None)
    if fused:
        x = rand((B, T, N * V + 2 * G * K + 8), seed + 4)
        s["v"], s["k"], s["q"] = (t.unflatten(2, (h, -1)) for t, h in
                                  ((x[:, :, :N * V], N), (x[:, :, N * V:N * V + G * K], G),
                                   (x[:, :, N * V + G * K:N * V + 2 * G * K], G)))
    else:
        s["q"], s["k"], s["v"] = rand((B, T, G, K), seed + 5), rand((B, T, G, K), seed + 6), rand((B, T, N, V), seed + 7)
    s["a"] = rand((B, T, N), seed + 8)
    return s


def oracle_inputs(s, absolute=False):
    d = {n: f64(s[n]) for n in ("q", "k", "v", "a", "alpha", "beta", "w_r", "H0")}
    if absolute:
        for n in ("q", "k", "v", "w_r", "H0"):
            d[n] = None if d[n] is None else np.abs(d[n])
    return d


def check_forward(s, y, H_T):
    want, states = ob.ssm_scan(**oracle_inputs(s))
    size, sizes = ob.ssm_scan(**oracle_inputs(s, True))
    within(y, want, 2.0 ** -8 * (np.abs(want) + size) + 1e-6, "y")
    within(H_T, states[-1], 2.0 ** -14 * sizes[-1] + 1e-7, "H_T")


@pytest.mark.parametrize("shape", SCAN)
@pytest.mark.parametrize("h0,fused", [(False, False), (True, True)])
def test_scan_forward(shape, h0, fused):
    s = scan_case(*shape, h0=h0, fused=fused)
    y, H_T = pkg.ssm_forward(s)
    check_forward(s, y, H_T)
    y2, H2, Hs = pkg.ssm_forward_train(s)
    assert torch.equal(y, y2) and torch.equal(H_T, H2)


@pytest.mark.parametrize("shape", SCAN)
@pytest.mark.parametrize("ends,fused", [(False, False), (True, True)])
def test_scan_backward(shape, ends, fused):
    """Every gradient; ``ends``: with an initial state and a gradient at the final one."""
    B, T, N, G, K, V = shape
    s = scan_case(*shape, seed=20, h0=ends, fused=fused)
    dy, dH = rand((B, T, N, V), 30), rand((B, N, K, V), 31, 0.5, torch.float32) if ends else None
    Hs = pkg.ssm_forward_train(s)[2]
    g = pkg.ssm_backward(s, Hs, dy, dH)
    want = ob.ssm_backward(**oracle_inputs(s), dy=f64(dy), dH_T=f64(dH))
    size = ob.ssm_backward(**oracle_inputs(s, True), dy=np.abs(f64(dy)), dH_T=None if dH is None else np.abs(f64(dH)), bound=True)
    for n in ("dq", "dk", "dv"):
        within(g[n], want[n], 2.0 ** -8 * (np.abs(want[n]) + size[n]) + 1e-6, n)
    within(g["da"], want["da"], 2.0 ** -8 * np.abs(want["da"]) + 2.0 ** -10 * size["da"].max() + 1e-6, "da")
    for n in ("dalpha", "dbeta", "dw_r", "dH0"):
        within(g[n], want[n], 2.0 ** -14 * size[n] + 1e-6, n)
    again = pkg.ssm_backward(s, Hs, dy, dH)
    assert all(torch.equal(g[n], again[n]) for n in g)


def test_scan_backward_is_the_directional_difference():
    """<gradient, direction> against a central difference of the fp64 oracle along it."""
    s = scan_case(1, 140, 2, 1, 64, 64, seed=40)
    dy = rand((1, 140, 2, 64), 41)
    g = pkg.ssm_backward(s, pkg.ssm_forward_train(s)[2], dy)
    d = oracle_inputs(s)
    r = np.random.default_rng(0)
    for n in ("q", "k", "v", "a", "alpha", "beta", "w_r", "H0"):
        u, eps = r.normal(size=d[n].shape), 1e-5
        loss = lambda e: float((ob.ssm_scan(**{**d, n: d[n] + e * u})[0] * f64(dy)).sum())  # noqa: E731
        num, got = (loss(eps) - loss(-eps)) / (2 * eps), float((f64(g["d" + n]) * u).sum())
        # a sum of rounded values: 2^-8 of the terms' root sum of squares, and the worst of them
        scale = np.sqrt((f64(g["d" + n]) ** 2 * u ** 2).sum()) + np.abs(f64(g["d" + n]) * u).max()
        assert abs(num - got) <= 2.0 ** -6 * scale + 1e-6 * abs(num), (n, num, got)


def test_scan_in_two_calls_is_one():
    """A prompt cut at an odd token, the state carried in place, against the oracle of the whole."""
    s = scan_case(2, 230, 3, 1, 64, 64, seed=50)
    cut = lambda lo, hi: {n: t[:, lo:hi] if n in ("q", "k", "v", "a") else t for n, t in s.items()}  # noqa: E731
    H = s["H0"].clone()
    ys = []
    for lo, hi in ((0, 101), (101, 101), (101, 230)):
        part = dict(cut(lo, hi), H0=H)
        ys.append(pkg.ssm_forward(part, H_T=H)[0])
    check_forward(s, torch.cat(ys, 1), H)


@pytest.mark.parametrize("shape", [(3, 9, 4, 2, 64, 64), (2, 5, 2, 1, 128, 128), (1, 4, 3, 3, 17, 33), (2, 3, 2, 1, 128, 64),
                                   (1, 3, 1, 1, 1, 1), (2, 4, 2, 2, 40, 24)])
def test_scan_tokens(shape):
    """Single tokens, state in place: fp32 arithmetic, so y is its bf16 rounding."""
    s = scan_case(*shape, seed=60)
    H, ys = s["H0"].clone(), []
    for t in range(shape[1]):
        tok = [s[n][:, t].contiguous() for n in ("q", "k", "v", "a")]
        y, out = pkg.ssm_step(*tok, s["alpha"], s["beta"], s["w_r"], H)
        assert out is H
        ys.append(y.unsqueeze(1))
    want, states = ob.ssm_scan(**oracle_inputs(s))
    size, sizes = ob.ssm_scan(**oracle_inputs(s, True))
    within(torch.cat(ys, 1), want, 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size + 1e-6)
    within(H, states[-1], 2.0 ** -18 * sizes[-1] + 1e-7)
    tok = [s[n][:, 0].contiguous() for n in ("q", "k", "v", "a")]
    y, H = pkg.ssm_step(*tok, s["alpha"], s["beta"], s["w_r"], None)
    want, states = ob.ssm_scan(**{**oracle_inputs({**s, "H0": None}), **{n: f64(s[n])[:, :1] for n in ("q", "k", "v", "a")}})
    within(H, states[1], 2.0 ** -18 * np.abs(states[1]) + 1e-7)


def test_scan_inert_and_resetting_tokens():
    """a = -infinity leaves the state as it is; a large a forgets it, exactly as f = 0 does."""
    s = scan_case(1, 150, 2, 1, 64, 64, seed=70)
    s["a"][:, 20:40] = -float("inf")
    s["a"][:, 64] = 200.0
    s["a"][:, 100] = 200.0
    s["k"][:, 64] = 0  # the resetting token itself adds nothing
    s["k"][:, 100] = 0
    y, H_T = pkg.ssm_forward(s)
    check_forward(s, y, H_T)
    late = {n: t[:, 101:] if n in ("q", "k", "v", "a") else t for n, t in s.items()}
    alone, H2 = pkg.ssm_forward(dict(late, H0=None))
    within(y[:, 101:], f64(alone), 2.0 ** -7 * ob.ssm_scan(**oracle_inputs(dict(late, H0=None), True))[0] + 1e-6)
    dy = rand((1, 150, 2, 64), 71)
    g = pkg.ssm_backward(s, pkg.ssm_forward_train(s)[2], dy)
    want = ob.ssm_backward(**oracle_inputs(s), dy=f64(dy))
    size = ob.ssm_backward(**oracle_inputs(s, True), dy=np.abs(f64(dy)), bound=True)
    assert float(g["da"][:, 20:40].float().abs().max()) == 0.0
    for n in ("dq", "dk", "dv"):
        within(g[n], want[n], 2.0 ** -8 * (np.abs(want[n]) + size[n]) + 1e-6, n)
    within(g["dH0"], want["dH0"], 2.0 ** -14 * size["dH0"] + 1e-6)


def test_scan_empty_sequence():
    s = scan_case(2, 0, 3, 1, 16, 24, seed=80)
    y, H_T, Hs = pkg.ssm_forward_train(s)
    assert y.shape == (2, 0, 3, 24) and torch.equal(H_T, s["H0"])
    dH = rand((2, 3, 16, 24), 81, 1.0, torch.float32)
    g = pkg.ssm_backward(s, Hs, torch.empty(2, 0, 3, 24, dtype=BF16, device=DEV), dH)
    assert torch.equal(g["dH0"], dH)
    assert all(float(g[n].abs().max()) == 0.0 for n in ("dalpha", "dbeta", "dw_r"))


def test_scan_runs_on_its_stream():
    s = scan_case(2, 700, 4, 1, 64, 64, seed=90)
    dy = rand((2, 700, 4, 64), 91)
    want = pkg.ssm_backward(s, pkg.ssm_forward_train(s)[2], dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _, _, Hs = pkg.ssm_forward_train(s, stream=side)
    got = pkg.ssm_backward(s, Hs, dy, stream=side)
    side.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)


def test_scan_replays_from_a_graph():
    s = scan_case(2, 300, 4, 2, 64, 64, seed=95)
    want, H = pkg.ssm_forward(s)
    pkg.ssm_step(*[s[n][:, 0].contiguous() for n in ("q", "k", "v", "a")], s["alpha"], s["beta"], s["w_r"], s["H0"].clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, H2 = pkg.ssm_forward(s)
    y.zero_(), H2.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(H, H2)


def test_scan_refuses_bad_tensors():
    s = scan_case(1, 8, 4, 2, 16, 16)
    with pytest.raises(ValueError):
        pkg.ssm_forward(dict(s, q=s["q"].repeat(1, 1, 2, 1)[:, :, :3], k=s["k"].repeat(1, 1, 2, 1)[:, :, :3]))
    with pytest.raises(TypeError):
        pkg.ssm_forward(dict(s, a=s["a"].float()))
    with pytest.raises(ValueError):
        pkg.ssm_forward(dict(s, v=s["v"].transpose(2, 3).contiguous().transpose(2, 3)))
    wide = scan_case(1, 8, 1, 1, 200, 16)
    with pytest.raises(binding.M2RNNError) as e:
        pkg.ssm_forward(wide)
    assert e.value.status == binding.ERR_UNSUPPORTED


# ---------------------------------------------------------------- gated group norm
NORM = [(1, 8, 1), (5, 64, 4), (7, 1024, 16), (3, 1000, 8), (33, 2048, 1), (2, 96, 32), (3, 9, 3), (2, 8192, 1),
        (2, 4097, 1), (4, 600, 2), (300, 1024, 16), (3, 130, 1), (2, 33, 1)]


def norm_case(rows, D, f32, gate, bias, seed=0):
    y = rand((rows, D), seed, 1.0, torch.float32 if f32 else BF16) + 0.5
    return (y, rand((rows, D), seed + 1, 1.5) if gate else None, 1.0 + rand((D,), seed + 2, 0.2, torch.float32),
            rand((D,), seed + 3, 0.2, torch.float32) if bias else None)


@pytest.mark.parametrize("rows,D,groups", NORM)
@pytest.mark.parametrize("f32,gate,bias", [(False, True, True), (True, True, False), (True, False, True), (False, False, False)])
def test_norm(rows, D, groups, f32, gate, bias):
    y, g, w, b = norm_case(rows, D, f32, gate, bias)
    out = pkg.gate_groupnorm(y, g, w, b, groups, 1e-5)
    want = ob.gate_groupnorm(f64(y), f64(g), f64(w), f64(b), groups, 1e-5)
    within(out, want, 2.0 ** -8 * np.abs(want) + 2e-5)
    dout = rand((rows, D), 9)
    got = pkg.gate_groupnorm_backward(y, g, w, b, dout, groups, 1e-5)
    ref = ob.gate_groupnorm_backward(f64(y), f64(g), f64(w), f64(b), f64(dout), groups, 1e-5)
    n, inv = ob._normalise(f64(y), groups, 1e-5)
    # each gradient is a combination of terms of at most inv * 8 in magnitude, a few 2^-22 off
    inv = np.repeat(inv[:, :, 0], D // groups, 1)
    within(got["dy"], ref["dy"], (0.0 if f32 else 2.0 ** -8) * np.abs(ref["dy"]) + 3e-5 * np.maximum(inv, 1.0), "dy")
    if gate:
        within(got["dg_pre"], ref["dg_pre"], 2.0 ** -8 * np.abs(ref["dg_pre"]) + 3e-5, "dg_pre")
    within(got["dw"], ref["dw"], 3e-6 * 8 * rows + 1e-6, "dw")
    within(got["dbias"], ref["dbias"], 3e-6 * 8 * rows + 1e-6, "dbias")


def test_norm_constant_group():
    """A group of equal values has no variance: its norm is zero, the output b SiLU(g)."""
    y, g, w, b = norm_case(4, 64, False, True, True)
    y[:, :16] = 3.0
    out = pkg.gate_groupnorm(y, g, w, b, 4, 1e-5)
    want = ob.gate_groupnorm(f64(y), f64(g), f64(w), f64(b), 4, 1e-5)
    within(out, want, 2.0 ** -8 * np.abs(want) + 2e-5)


def test_norm_unaligned_and_empty():
    base = rand((5 * 64 + 1,), 3)
    y = base[1:].view(5, 64)
    w = 1.0 + rand((64,), 4, 0.2, torch.float32)
    want = ob.gate_groupnorm(f64(y), None, f64(w), None, 2, 1e-5)
    within(pkg.gate_groupnorm(y, None, w, None, 2, 1e-5), want, 2.0 ** -8 * np.abs(want) + 2e-5)
    assert pkg.gate_groupnorm(y[:0], None, w, None, 2).shape == (0, 64)
    g = pkg.gate_groupnorm_backward(y[:0], None, w, None, y[:0], 2)
    assert float(g["dw"].abs().max()) == 0.0


# ---------------------------------------------------------------- chunk edges, shared heads, many rows
# Lengths around the scan's chunks of 128 tokens, many heads on one q and k (whose gradients are summed
# over parts), more pairs than SMs, widths on either side of a tile of 64.
EDGES = [(1, 127, 2, 1, 64, 64), (2, 128, 2, 2, 128, 64), (1, 255, 3, 1, 64, 128), (1, 256, 2, 1, 128, 128),
         (1, 257, 2, 1, 40, 72), (1, 385, 6, 2, 65, 65), (1, 700, 40, 1, 64, 64), (2, 513, 5, 1, 128, 64),
         (4, 130, 48, 3, 64, 64), (1, 1, 160, 160, 128, 128)]


@pytest.mark.parametrize("shape", EDGES)
@pytest.mark.parametrize("ends", [False, True])
def test_scan_chunk_edges(shape, ends):
    test_scan_forward(shape, ends, not ends)
    test_scan_backward(shape, ends, not ends)
    assert pkg.stream_status() == 0


@pytest.mark.parametrize("shape", [(1, 1100, 2, 1, 64, 64), (1, 4217, 4, 2, 64, 64), (1, 2600, 3, 1, 128, 128)])
def test_scan_segments_of_several_pieces(shape):
    """Few pairs: segments whose states are found in three or four pieces each, the last segment shorter
    than its pieces."""
    test_scan_forward(shape, True, False)
    test_scan_backward(shape, True, False)
    assert pkg.stream_status() == 0


def test_scan_long_decays_between_chunks():
    """Decays of one token from none to complete (f from 1 to 0), over chunks and pieces."""
    s = scan_case(1, 1500, 2, 1, 64, 64, seed=101)
    s["a"] = (rand((1, 1500, 2), 102, 12.0, torch.float32)).to(BF16)
    check_forward(s, *pkg.ssm_forward(s))


def test_norm_many_rows():
    """Enough short groups for two rows a team, an odd number of them."""
    test_norm(4867, 1024, 16, False, True, True)


def test_conv_long_stretches():
    """Stretches of several tens of tokens a thread, the last cut inside a group of loads."""
    test_conv_window((3, 4099, 256), True, True, 8)
    test_conv_backward((3, 4099, 256), True, 8)


def block_f64(block, x):
    """The example's block from its formulas, in double precision on the CPU, with autograd."""
    p = {n: t.detach().double().cpu().requires_grad_() for n, t in block.p.items()}
    x = x.double().cpu().requires_grad_()
    N, G, K, V, C = block.N, block.G, block.K, block.V, block.C
    B, T, _ = x.shape
    z = x @ p["w_in"].T
    gate, u, a = z[..., :N * V], z[..., N * V:N * V + C], z[..., N * V + C:N * V + C + N]
    X = torch.cat([u.new_zeros(B, 3, C), u], 1)
    c = torch.nn.functional.silu(p["conv_b"] + sum(X[:, j:j + T] * p["conv_w"][:, j] for j in range(4)))
    v = c[..., :N * V].unflatten(-1, (N, V))
    k, q = (t.unflatten(-1, (G, K)).repeat_interleave(N // G, 2) for t in c[..., N * V:].chunk(2, -1))
    d = torch.nn.functional.softplus(a + p["beta"])
    f = torch.exp(-p["alpha"] * d)
    H, ys = x.new_zeros(B, N, K, V), []
    for t in range(T):
        H = f[:, t, :, None, None] * H + (d[:, t, :, None] * k[:, t])[..., None] * v[:, t, :, None]
        ys.append((H * q[:, t, ..., None]).sum(-2) + p["w_r"] * v[:, t])
    n = torch.nn.functional.layer_norm(torch.stack(ys, 1), (V,), eps=1e-5).flatten(2)
    return ((n * p["norm_w"] + p["norm_b"]) * torch.nn.functional.silu(gate)) @ p["w_out"].T, p, x


def test_block_gradients():
    """The three operators together, forward and backward, against double precision.  At most eight
    intermediates between a parameter and its gradient are bf16 (2^-9 of each value), and no stage
    here more than doubles a relative error: 8 x 2 x 2^-9 = 2^-5 of the gradient's norm."""
    from examples.ssm_block import Block
    block, x, dout = Block(seed=3), rand((2, 200, 256), 130), rand((2, 200, 256), 131)
    out, g = block.train(x, dout)
    want, p, x64 = block_f64(block, x)
    (want * dout.double().cpu()).sum().backward()
    grads = dict({n: t.grad for n, t in p.items()}, x=x64.grad)
    assert float((out.double().cpu() - want.detach()).norm()) <= 2.0 ** -5 * float(want.detach().norm())
    for n, ref in grads.items():
        assert float((g[n].double().cpu() - ref).norm()) <= 2.0 ** -5 * float(ref.norm()), n


def test_block_example():
    """Prompts in parts and tokens agree with one call: outputs are bf16 of sums of 384 products of
    values that each call rounds alike but for the chunks' cuts, 2^-7 at most, within 2^-5 of the
    largest; and steps of a thousandth of each parameter along its gradient lower the loss."""
    from examples.ssm_block import check
    split, losses = check()
    assert split < 2.0 ** -5 and all(b < a for a, b in zip(losses, losses[1:])), (split, losses)


def test_offsets_beyond_32_bits():
    """Tensors of more than 2^31 values: their ends against calls on the ends alone.  Conv and norm do
    not look back that far, so they give the same bits; the scan's cut is on a chunk, and only the pieces
    of the sequence, and with them float32 roundings of the state, differ: a bf16 rounding apart."""
    T, C = 1_100_000, 2048
    tail = T - (T - 12_000) // 128 * 128  # the cut is at a chunk's edge
    x = torch.randn(1, T, C, device=DEV, dtype=BF16)
    w, b = rand((C, 4), 1, 0.6, torch.float32), rand((C,), 2, 0.3, torch.float32)
    last = x[:, -tail:].contiguous()
    out, window = pkg.conv_silu_window(x, w, b)
    end, _ = pkg.conv_silu_window(last, w, b, x[:, -tail - 3:-tail].contiguous())
    assert torch.equal(out[:, -tail:], end) and torch.equal(window, x[:, -3:])
    y = pkg.gate_groupnorm(x[0], out[0], b.abs() + 0.5, None, 32)
    assert torch.equal(y[-tail:], pkg.gate_groupnorm(last[0], end[0], b.abs() + 0.5, None, 32))
    del out, y
    s = scan_case(1, T, 32, 1, 64, 1, seed=140, h0=False)
    s.update(v=x.view(1, T, 32, 64), w_r=rand((32, 64), 141, 1.0, torch.float32))
    cut = lambda lo, hi: {n: t[:, lo:hi] if n in ("q", "k", "v", "a") else t for n, t in s.items()}  # noqa: E731
    y, H = pkg.ssm_forward(s)
    before = pkg.ssm_forward(cut(0, T - tail))[1]
    end, H_end = pkg.ssm_forward(dict(cut(T - tail, T), H0=before))
    assert float((y[:, -tail:].float() - end.float()).abs().max()) <= 2.0 ** -7 * float(end.float().abs().max())
    assert float((H - H_end).abs().max()) <= 2.0 ** -14 * float(H.abs().max())
    assert pkg.stream_status() == 0
