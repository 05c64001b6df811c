"""The binding of the selective block without a GPU: what it refuses before any call into the library.

Tensors are stand-ins with the attributes that the checks read; the library is a stub that fails the
test when it is reached.
"""
import contextlib
from types import SimpleNamespace

import pytest
import torch

import matrix_state_nonlinear_gb300 as pkg
from matrix_state_nonlinear_gb300 import ssm


class Fake:
    """A dense CUDA tensor's attributes."""

    def __init__(self, dev, *shape, dtype=torch.bfloat16):
        self.is_cuda, self.dev, self.shape, self.dtype = True, dev, torch.Size(shape), dtype
        self.device = torch.device("cuda", dev)

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def stride(self, i=None):
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s) if i is None else s[i]

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 1 << 20

    def new_empty(self, shape):
        return Fake(self.dev, *shape, dtype=self.dtype)


def calls(dev, B=2, T=5, C=8, N=2, K=16, V=16):
    """Every entry with well-formed arguments on one device."""
    f32 = torch.float32
    t = lambda *s, dtype=torch.bfloat16: Fake(dev, *s, dtype=dtype)  # noqa: E731
    s = dict(q=t(B, T, N, K), k=t(B, T, N, K), v=t(B, T, N, V), a=t(B, T, N), alpha=t(N, dtype=f32), beta=t(N, dtype=f32),
             w_r=t(N, V, dtype=f32))
    w, bias = t(C, 4, dtype=f32), t(C, dtype=f32)
    x, win, token = t(B, T, C), t(B, 3, C), t(B, C)
    return {
        "conv_silu_window": lambda **kw: pkg.conv_silu_window(x, w, bias, win, out=x, window_out=win, **kw),
        "conv_silu_step": lambda **kw: pkg.conv_silu_step(token, w, bias, win, out=token, **kw),
        "conv_silu_backward": lambda **kw: pkg.conv_silu_backward(x, w, bias, x, win, workspace=x, **kw),
        "ssm_forward": lambda **kw: pkg.ssm_forward(s, y=s["v"], H_T=t(B, N, K, V, dtype=f32), workspace=x, **kw),
        "ssm_forward_train": lambda **kw: pkg.ssm_forward_train(s, Hs=t(64, dtype=torch.uint8), workspace=x, **kw),
        "ssm_backward": lambda **kw: pkg.ssm_backward(s, t(64, dtype=torch.uint8), s["v"], workspace=x, **kw),
        "ssm_step": lambda **kw: pkg.ssm_step(t(B, N, K), t(B, N, K), t(B, N, V), t(B, N), s["alpha"], s["beta"], s["w_r"],
                                              t(B, N, K, V, dtype=f32), y=t(B, N, V), **kw),
        "gate_groupnorm": lambda **kw: pkg.gate_groupnorm(token, token, bias, bias, 2, out=token, **kw),
        "gate_groupnorm_backward": lambda **kw: pkg.gate_groupnorm_backward(token, token, bias, bias, token, 2, workspace=x,
                                                                            **kw),
    }


NAMES = sorted(calls(0))


class Reached(Exception):
    pass


@pytest.fixture
def library(monkeypatch):
    """A library of which every function raises Reached with its arguments; device 0 is current."""
    state = SimpleNamespace(current=0)

    class Stub:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_bytes"):
                    return 64
                raise Reached(name, args)
            return call

    @contextlib.contextmanager
    def on(stream):
        before, state.current = state.current, stream.device.index
        yield
        state.current = before

    monkeypatch.setattr(ssm, "load_library", Stub)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state.current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "stream", on)
    return state


@pytest.mark.parametrize("name", NAMES)
def test_well_formed_calls_reach_the_library(library, name):
    with pytest.raises(Reached):
        calls(0)[name]()
    library.current = 1
    with pytest.raises(Reached):
        calls(1)[name]()


@pytest.mark.parametrize("name", NAMES)
def test_another_device_is_refused(library, name):
    """Tensors of cuda:1 while cuda:0 is current would be read by kernels on cuda:0."""
    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
        calls(1)[name]()


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(library, name):
    stream = SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
        calls(0)[name](stream=stream)
    with pytest.raises(Reached):  # the stream's own device, whichever is current
        calls(1)[name](stream=stream)


@pytest.mark.parametrize("offset", [4, 8, 12])
def test_taps_off_16_bytes_are_refused_by_name(library, offset):
    """As a view into a flat buffer of parameters may have them."""
    class At(Fake):
        def data_ptr(self):
            return (1 << 20) + offset
    w, x, win = At(0, 8, 4, dtype=torch.float32), Fake(0, 2, 5, 8), Fake(0, 2, 3, 8)
    for call in (lambda: pkg.conv_silu_window(x, w, None, win, out=x, window_out=win),
                 lambda: pkg.conv_silu_step(Fake(0, 2, 8), w, None, win, out=Fake(0, 2, 8)),
                 lambda: pkg.conv_silu_backward(x, w, None, x, win, workspace=x)):
        with pytest.raises(ValueError, match="w: must be 16-byte aligned"):
            call()


def test_a_first_token_gets_a_window(library):
    """conv_silu_step without a window starts from zeros and returns the one after the token."""
    with pytest.raises(Reached) as e:
        pkg.conv_silu_step(Fake(0, 2, 8), Fake(0, 8, 4, dtype=torch.float32), None, None, out=Fake(0, 2, 8))
    _, args = e.value.args
    assert args[3] is None and args[5] is not None
