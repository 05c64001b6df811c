"""The selective block's calls run where they are told to, all their launches.

Both tests fail if any launch of a call goes to another stream: the first reads inputs that arrive late
on the call's own stream, the second replays a captured call on inputs that came after the capture.
"""
import pytest
import torch

import matrix_state_nonlinear_gb300 as pkg
from test_ssm_gpu import built, conv_case, norm_case, rand, scan_case  # noqa: F401

pytestmark = pytest.mark.gpu


def scan(shape, seed):
    s = scan_case(*shape, seed=seed)
    B, T, N, _, K, V = shape
    return dict(s, dy=rand((B, T, N, V), seed + 50), dH=rand((B, N, K, V), seed + 51, 0.5, torch.float32))


def train(s, **kw):
    y, H, Hs = pkg.ssm_forward_train(s, **kw)
    return [y, H, *pkg.ssm_backward(s, Hs, s["dy"], s["dH"], **kw).values()]


def named(names, tensors):
    return {n: t for n, t in zip(names, tensors) if t is not None}


# A call of the package: its inputs from a seed, and the outputs of one pass on them.
CALLS = {
    "conv": (lambda seed: named(("x", "w", "bias", "window"), conv_case(2, 300, 40, seed)),
             lambda s, **kw: list(pkg.conv_silu_window(*s.values(), **kw))),
    "conv step": (lambda seed: named(("x", "w", "bias", "window"), [t[:, 0] if i == 0 else t for i, t in
                                                                    enumerate(conv_case(64, 1, 40, seed))]),
                  lambda s, **kw: list(pkg.conv_silu_step(*s.values(), window_out=torch.empty_like(s["window"]), **kw))),
    "conv backward": (lambda seed: dict(named(("x", "w", "bias", "window"), conv_case(2, 300, 40, seed)), dout=rand((2, 300, 40), seed + 9)),
                      lambda s, **kw: list(pkg.conv_silu_backward(s["x"], s["w"], s["bias"], s["dout"], s["window"], **kw).values())),
    # segments of several pieces, heads' gradients summed over parts
    "scan": (lambda seed: scan((1, 2600, 3, 1, 128, 128), seed), lambda s, **kw: list(pkg.ssm_forward(s, **kw))),
    "scan train": (lambda seed: scan((1, 2600, 3, 1, 128, 128), seed), train),
    "scan train, whole sequences": (lambda seed: scan((2, 300, 80, 4, 64, 64), seed), train),
    "scan train, odd widths": (lambda seed: scan((1, 700, 2, 1, 33, 17), seed), train),
    "scan step": (lambda seed: {n: t[:, 0].contiguous() if n in "qkva" else t for n, t in scan_case(9, 1, 4, 2, 64, 64, seed).items()},
                  lambda s, **kw: list(pkg.ssm_step(*(s[n] for n in ("q", "k", "v", "a", "alpha", "beta", "w_r", "H0")),
                                                    H_out=torch.empty_like(s["H0"]), **kw))),
    "norm": (lambda seed: named(("y", "g_pre", "w", "bias"), norm_case(300, 1024, False, True, True, seed)),
             lambda s, **kw: [pkg.gate_groupnorm(*s.values(), 16, **kw)]),
    "norm backward": (lambda seed: dict(named(("y", "g_pre", "w", "bias"), norm_case(300, 1024, False, True, True, seed)),
                                        dout=rand((300, 1024), seed + 9)),
                      lambda s, **kw: list(pkg.gate_groupnorm_backward(*s.values(), 16, **kw).values())),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_on_a_side_stream(name):
    """The inputs arrive on the side stream after some 50 ms of waiting there; a launch on any other
    stream would have run on the zeros that were there before."""
    make, run = CALLS[name]
    new = make(400)
    want = run(new)
    late = {n: torch.zeros_like(t) for n, t in new.items()}
    run(late)  # (loads every kernel)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        for n, t in new.items():
            late[n].copy_(t)
    got = run(late, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert pkg.stream_status() == 0


@pytest.mark.parametrize("name", sorted(CALLS))
def test_replays_from_a_graph(name):
    """Captured on some inputs, replayed on others: the bits of a call on those."""
    make, run = CALLS[name]
    s, new = make(410), make(420)
    run(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(s)
    want = run(new)
    for _ in range(2):
        for t in got:
            t.zero_()
        for n, t in new.items():
            s[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert pkg.stream_status() == 0
