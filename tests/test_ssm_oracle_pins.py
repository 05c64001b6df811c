"""The selective block's oracle against closed forms and central differences, and the entry
points' refusals (no GPU: every call here is rejected before anything is enqueued)."""
import ctypes

import numpy as np
import pytest
import torch

import __graft_entry__
import matrix_state_nonlinear_gb300 as pkg
from matrix_state_nonlinear_gb300 import m2rnn as binding
from oracle import ssm_block as ob


def scan_inputs(seed=0, B=2, T=5, N=4, G=2, K=3, V=2):
    r = np.random.default_rng(seed)
    return dict(q=r.normal(size=(B, T, G, K)), k=r.normal(size=(B, T, G, K)), v=r.normal(size=(B, T, N, V)),
                a=r.normal(size=(B, T, N)), alpha=r.uniform(0.1, 2, N), beta=r.normal(size=N),
                w_r=r.normal(size=(N, V)), H0=r.normal(size=(B, N, K, V)))


def differences(f, x, eps=1e-6):
    """Central differences of the scalar f at every entry of x."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        old = x[i]
        x[i] = old + eps
        up = f()
        x[i] = old - eps
        g[i] = (up - f()) / (2 * eps)
        x[i] = old
    return g


def test_scan_closed_forms():
    s = scan_inputs()
    s["a"][:] = -np.inf  # inert tokens: d = 0, f = 1
    y, states = ob.ssm_scan(**s)
    assert np.array_equal(states[-1], s["H0"])
    s = scan_inputs(N=1, G=1)
    s["alpha"][:] = 0.0  # f = 1: the state is the sum of its outer products
    y, states = ob.ssm_scan(**s)
    d = np.log1p(np.exp(s["a"] + s["beta"]))
    want = s["H0"][:, 0] + np.einsum("bt,btk,btv->bkv", d[..., 0], s["k"][:, :, 0], s["v"][:, :, 0])
    assert np.allclose(states[-1][:, 0], want, rtol=1e-12)


def test_scan_gradients_are_differences():
    s = scan_inputs(1)
    r = np.random.default_rng(2)
    dy, dH = r.normal(size=(2, 5, 4, 2)), r.normal(size=(2, 4, 3, 2))

    def loss():
        y, states = ob.ssm_scan(**s)
        return (y * dy).sum() + (states[-1] * dH).sum()

    g = ob.ssm_backward(**s, dy=dy, dH_T=dH)
    for name, x in s.items():
        assert np.allclose(g["d" + name], differences(loss, x), rtol=1e-6, atol=1e-8), name


@pytest.mark.parametrize("T", [1, 2, 5])
def test_conv_gradients_are_differences(T):
    r = np.random.default_rng(3)
    s = dict(x=r.normal(size=(2, T, 3)), w=r.normal(size=(3, 4)), bias=r.normal(size=3), window=r.normal(size=(2, 3, 3)))
    dout = r.normal(size=(2, T, 3))
    g = ob.conv_window_backward(**s, dout=dout)
    for name, x in s.items():
        assert np.allclose(g["d" + name], differences(lambda: (ob.conv_window(**s)[0] * dout).sum(), x), rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("gate", [True, False])
def test_norm_gradients_are_differences(gate):
    r = np.random.default_rng(4)
    s = dict(y=r.normal(size=(2, 6)), g=r.normal(size=(2, 6)) if gate else None, w=r.normal(size=6), bias=r.normal(size=6))
    dout = r.normal(size=(2, 6))
    g = ob.gate_groupnorm_backward(**s, dout=dout, groups=2, eps=1e-5)
    for name, key in (("y", "dy"), ("g", "dg_pre"), ("w", "dw"), ("bias", "dbias")):
        if s[name] is not None:
            num = differences(lambda: (ob.gate_groupnorm(**s, groups=2, eps=1e-5) * dout).sum(), s[name])
            assert np.allclose(g[key], num, rtol=1e-6, atol=1e-7), name


# ---------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return binding.load_library()


ONE = ctypes.c_void_p(1 << 20)  # never read: every call below is refused first


def forward(lib, B=1, T=4, N=2, G=1, K=8, V=8, ws=ONE, ws_bytes=1 << 30, strides=None, alpha=ONE, y=ONE, Hs=None):
    return lib.m2rnn_ssm_forward_bf16(ONE, ONE, ONE, ONE, alpha, ONE, ONE, None, y, None, Hs, strides, B, T, N, G, K, V,
                                      ws, ws_bytes, None)


def test_scan_refusals(lib):
    bad, wide = binding.ERR_INVALID_ARG, binding.ERR_UNSUPPORTED
    assert forward(lib, B=0) == bad and forward(lib, T=-1) == bad and forward(lib, N=3, G=2) == bad
    assert forward(lib, G=0) == bad and forward(lib, K=0) == bad
    assert forward(lib, K=129) == wide and forward(lib, V=129) == wide
    assert forward(lib, alpha=None) == bad and forward(lib, y=None) == bad
    assert forward(lib, Hs=ctypes.c_void_p(8)) == bad
    assert forward(lib, strides=(ctypes.c_longlong * 8)(-1, *[1] * 7)) == bad
    need = lib.m2rnn_ssm_workspace_bytes(1, 4, 2, 1, 8, 8, 1)
    args = [ONE] * 7 + [ONE, ONE, None] + [ONE] * 7 + [None, None, 1, 4, 2, 1, 8, 8]
    assert lib.m2rnn_ssm_backward_bf16(*args, ONE, need - 1, None) == bad
    assert lib.m2rnn_ssm_backward_bf16(*args, None, need, None) == bad
    assert lib.m2rnn_ssm_workspace_bytes(1, 4, 3, 2, 8, 8, 0) == 0
    assert lib.m2rnn_ssm_states_bytes(2, 129, 3, 4, 5) == 4 * 2 * 3 * 3 * 4 * 5
    assert lib.m2rnn_ssm_step_bf16(*[ONE] * 8, None, ONE, 1, 2, 1, 8, 8, None) == bad
    assert lib.m2rnn_ssm_step_bf16(*[ONE] * 10, 1, 2, 1, 8, 200, None) == wide


def test_conv_and_norm_refusals(lib):
    bad, wide = binding.ERR_INVALID_ARG, binding.ERR_UNSUPPORTED
    conv = lib.m2rnn_conv_silu_window_bf16
    assert conv(ONE, None, None, None, ONE, None, 1, 1, 8, 8, 8, None) == bad
    assert conv(None, ONE, None, None, ONE, None, 1, 1, 8, 8, 8, None) == bad
    assert conv(ONE, ctypes.c_void_p(4), None, None, ONE, None, 1, 1, 8, 8, 8, None) == bad
    assert conv(ONE, ONE, None, None, ONE, None, 1, 1, 8, -8, 8, None) == bad
    need = lib.m2rnn_conv_silu_backward_workspace_bytes(1, 9, 8)
    assert need > 0
    assert lib.m2rnn_conv_silu_backward_bf16(*[ONE] * 9, 1, 9, 8, 72, 8, ONE, need - 1, None) == bad
    norm = lib.m2rnn_gate_groupnorm
    assert norm(ONE, 0, ONE, ONE, None, 1e-5, ONE, 4, 10, 3, None) == bad
    assert norm(ONE, 0, ONE, ONE, None, -1.0, ONE, 4, 10, 2, None) == bad
    assert norm(ONE, 0, ONE, ONE, None, float("nan"), ONE, 4, 10, 2, None) == bad
    assert norm(ONE, 0, ONE, ONE, None, 1e-5, ONE, 4, 20000, 2, None) == wide
    assert norm(None, 0, ONE, ONE, None, 1e-5, None, 0, 10, 2, None) == binding.OK  # no rows: nothing to do
    need = lib.m2rnn_gate_groupnorm_backward_workspace_bytes(4, 16, 2)
    back = lib.m2rnn_gate_groupnorm_backward
    assert back(ONE, 0, ONE, ONE, None, 1e-5, ONE, ONE, None, ONE, ONE, 4, 16, 2, ONE, need, None) == bad  # a gate without dg
    assert back(ONE, 0, ONE, ONE, None, 1e-5, ONE, ONE, ONE, ONE, ONE, 4, 16, 2, ONE, need - 1, None) == bad


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pkg.conv_silu_window(x, torch.zeros(8, 4))
    with pytest.raises(ValueError):
        pkg.gate_groupnorm(x, None, torch.ones(8))
    with pytest.raises(ValueError):
        pkg.ssm_forward(dict(q=x.unsqueeze(2), k=x.unsqueeze(2), v=x.unsqueeze(2), a=x[:, :, :1]))
