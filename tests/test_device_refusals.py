"""The recurrence's binding refuses tensors of another device than the current one, on which its kernels
would launch; without a GPU, with stand-ins for tensors and a stub of the library."""
import pytest
import torch

import matrix_state_nonlinear_gb300 as pkg
from matrix_state_nonlinear_gb300 import m2rnn as binding
from test_ssm_binding import Fake


class Reached(Exception):
    pass


class Stub:
    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                return 64
            raise Reached(name)
        return call


def calls(dev, B=2, T=5, N=2, K=16, V=16, C=16):
    f32, bf = torch.float32, torch.bfloat16
    t = lambda *s, dtype=bf: Fake(dev, *s, dtype=dtype)  # noqa: E731
    y, H = t(B, T, N, V, dtype=f32), t(B, N, K, V, dtype=f32)

    def inputs(op):
        return dict(q=t(B, T, N, K, dtype=op), k=t(B, T, N, K, dtype=op), v=t(B, T, N, V, dtype=op), a=t(B, T, N, dtype=op),
                    alpha=t(N, dtype=f32), beta=t(N, dtype=f32), W=t(N, V, V, dtype=op), w_r=t(N, V, dtype=f32))
    grads = dict(dq=t(B, T, N, K, dtype=f32), dk=t(B, T, N, K, dtype=f32), dv=y, da=t(B, T, N, dtype=f32), dalpha=t(N, dtype=f32),
                 dbeta=t(N, dtype=f32), dW=t(N, V, V, dtype=f32), dw_r=t(N, V, dtype=f32), dH0=H)
    s, Hs = inputs(bf), t(B, N, T, K, V)
    taps = {w + n: t(N * d, 4, dtype=f32) if w == "w" else t(N * d, dtype=f32) for w in "wb" for n, d in zip("qkv", (K, K, V))}
    return {
        "forward_f32": lambda st: pkg.m2rnn_forward(inputs(f32), y, H, stream=st),
        "forward_bf16": lambda st: pkg.m2rnn_forward(s, y, H, stream=st),
        "forward_conv": lambda st: binding.m2rnn_forward_conv(s, taps, y, H, stream=st),
        "forward_train": lambda st: pkg.m2rnn_forward_train(s, y, H, Hs, stream=st),
        "backward": lambda st: pkg.m2rnn_backward(s, Hs, y, grads=grads, workspace=Hs, stream=st),
        "backward_noalloc": lambda st: binding.m2rnn_backward_noalloc(s, Hs, y, grads=grads, stream=st),
        "decode_step": lambda st: pkg.m2rnn_decode_step(t(B, N, K), t(B, N, K), t(B, N, V), t(B, N), s["alpha"], s["beta"],
                                                        s["W"], s["w_r"], H, y=t(B, N, V, dtype=f32), stream=st),
        "conv_silu": lambda st: pkg.conv_silu(t(B, T, C), t(C, 4, dtype=f32), None, t(B, T, C), stream=st),
        "gate_rmsnorm": lambda st: pkg.gate_rmsnorm(y, t(B, T, N, V), t(V, dtype=f32), out=t(B, T, N, V), stream=st),
    }


@pytest.mark.parametrize("name", sorted(calls(0)))
def test_another_device_is_refused(monkeypatch, name):
    class Stream:
        cuda_stream = 0
    monkeypatch.setattr(binding, "load_library", Stub)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    with pytest.raises(Reached):
        calls(0)[name](Stream)
    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
        calls(1)[name](Stream)
