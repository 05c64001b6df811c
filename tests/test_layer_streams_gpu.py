"""The calls of the residual norm, the 8-bit product and the clip run where they are told to, all their
launches; they can be captured into a graph, and calls at once do not meet.

As in the selective block's test: the first test reads inputs that arrive late on the call's own stream, the
second replays a captured call on inputs that came after the capture.
"""
import pytest
import torch

import matrix_state_nonlinear_gb300 as pkg
from test_layer_gpu import BF16, F32, built, linear_case, norm_case, rand  # noqa: F401

pytestmark = pytest.mark.gpu


def norms(rows, D, f32, seed):
    x, r, w = norm_case(rows, D, f32, True, seed)
    return dict(x=x.contiguous(), residual=r.contiguous(), w=w)


def linears(M, N, K, seed):
    return dict(zip(("q", "s", "w", "sw"), linear_case(M, N, K, seed)))


def raws(M, N, K, seed):
    s = linears(M, N, K, seed)
    return dict(x=rand((M, K), seed + 7), w=s["w"], sw=s["sw"])


def clips(seed):
    return {f"g{i}": rand((n,), seed + i, 1.0, BF16 if i % 2 else F32) for i, n in enumerate((70000, 31, 5000, 200001, 8))}


def clip_out(s, **kw):
    out = [torch.empty_like(t) for t in s.values()]
    norm = pkg.clip_grad_norm(s, 0.5, out=out, **kw)
    return [norm, *out]


def plain(s):  # torch's 8-bit types have few operators: as bytes
    return s.view(torch.uint8) if s.dtype.itemsize == 1 else s


CALLS = {
    "norm": (lambda seed: norms(300, 1024, False, seed), lambda s, **kw: list(pkg.add_rmsnorm(*s.values(), **kw))),
    "norm 8 bits": (lambda seed: norms(300, 1000, True, seed), lambda s, **kw: list(pkg.add_rmsnorm_fp8(*s.values(), **kw))),
    "norm backward": (lambda seed: dict(h=rand((3000, 520), seed), w=rand((520,), seed + 1, 1.0, F32), dout=rand((3000, 520), seed + 2),
                                        dh=rand((3000, 520), seed + 3)),
                      lambda s, **kw: list(pkg.add_rmsnorm_backward(*s.values(), **kw).values())),
    "quantise": (lambda seed: dict(x=rand((300, 1000), seed)), lambda s, **kw: list(pkg.quantise_fp8(s["x"], **kw))),
    "quantise weight": (lambda seed: dict(w=rand((300, 1000), seed)), lambda s, **kw: list(pkg.quantise_weight_fp8(s["w"], **kw))),
    "linear, K split": (lambda seed: linears(50, 300, 2000, seed), lambda s, **kw: [pkg.linear_fp8(*s.values(), **kw)]),
    "linear, pairs": (lambda seed: linears(2100, 2200, 300, seed), lambda s, **kw: [pkg.linear_fp8(*s.values(), **kw)]),
    "linear, quantised on the way": (lambda seed: raws(3, 300, 2000, seed), lambda s, **kw: [pkg.linear_fp8(s["x"], None, s["w"], s["sw"], **kw)]),
    "linear, quantised before": (lambda seed: raws(70, 300, 2000, seed), lambda s, **kw: [pkg.linear_fp8(s["x"], None, s["w"], s["sw"], **kw)]),
    "clip": (clips, clip_out),
    "norm of gradients": (clips, lambda s, **kw: [pkg.grad_norm(s, **kw)]),
}


def copy(to, new):
    for n in to:
        plain(to[n]).copy_(plain(new[n]))


def zero(s):
    for t in s.values():
        plain(t).zero_()


def same(got, want):
    return all(torch.equal(plain(a), plain(b)) for a, b in zip(got, want))


@pytest.mark.parametrize("name", sorted(CALLS))
def test_on_a_side_stream(name):
    """The inputs arrive on the side stream after some 50 ms of waiting there; a launch on any other stream
    would have run on the zeros that were there before."""
    make, run = CALLS[name]
    new = make(400)
    want = run(new)
    s = make(400)
    zero(s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        copy(s, new)
    got = run(s, stream=side)
    side.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_captured(name):
    """A graph's replay computes on the inputs that are there when it runs, twice the same."""
    make, run = CALLS[name]
    s, new = make(500), make(501)
    run(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = run(s)
    for inputs in (new, make(502), new):
        want = run(inputs)
        copy(s, inputs)
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_two_at_once(name):
    """Calls on two streams at once, many times over, give the bits of one alone."""
    make, run = CALLS[name]
    a, b = make(600), make(601)
    want = run(a), run(b)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(8):
        got.append((run(a, stream=streams[0]), run(b, stream=streams[1])))
    torch.cuda.synchronize()
    assert all(same(x, want[0]) and same(y, want[1]) for x, y in got)
    assert pkg.stream_status() == 0
