"""C entries of the layer refuse addresses off their type's boundary, which a kernel would fault on.  No GPU: the
addresses are never read."""
import ctypes

import pytest

import __graft_entry__
from matrix_state_nonlinear_gb300 import m2rnn as binding

A, INVALID = 1 << 20, binding.ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return binding.load_library()


def norm(lib, f32, **at):
    a = dict(dict(x=A, stream=A, w=A, h=A, out=A), **at)
    return lib.m2rnn_add_rmsnorm(a["x"], 8, a["stream"], f32, 8, a["w"], 1e-5, a["h"], a["out"], 4, 8, None)


def norm_fp8(lib, f32, **at):
    a = dict(dict(x=A, stream=A, w=A, h=A), **at)
    return lib.m2rnn_add_rmsnorm_fp8(a["x"], 8, a["stream"], f32, 8, a["w"], 1e-5, a["h"], A, 16, A, 4, 8, None)


def backward(lib, f32, **at):
    a = dict(dict(h=A, w=A, dout=A, dh=A, dx=A, dresidual=A, dw=A), **at)
    return lib.m2rnn_add_rmsnorm_backward(a["h"], f32, a["w"], 1e-5, a["dout"], a["dh"], a["dx"], a["dresidual"], a["dw"], 4, 8, A, 1 << 20,
                                          None)


def quantise(lib, f32, **at):
    return lib.m2rnn_quantise_fp8(at["x"], f32, 8, A, 16, A, 4, 8, None)


def quantise_weight(lib, f32, **at):
    return lib.m2rnn_quantise_weight_fp8(at["w"], f32, 8, A, 16, A, 4, 8, None)


def linear(lib, f32, **at):
    return lib.m2rnn_linear_fp8(A, 16, A, A, 16, A, at["out"], f32, 4, 8, 8, None)


def linear_quantise(lib, f32, **at):
    a = dict(dict(x=A, out=A), **at)
    return lib.m2rnn_linear_quantise_fp8(a["x"], f32, 8, A, 16, A, a["out"], f32, 4, 8, 8, A, 1 << 20, None)


def clip(lib, f32, **at):
    kept = [ctypes.c_uint64(A), ctypes.c_uint64(A), ctypes.c_longlong(4), ctypes.c_ubyte(f32)]
    return lib.m2rnn_clip_grad_norm(*map(ctypes.addressof, kept), 1, 1.0, at["norm"], A, 1 << 20, None)


WIDE, HALF, FLOAT = "of the stream's type", "bf16", "float32"
CALLS = [(norm, dict(x=HALF, stream=WIDE, w=FLOAT, h=WIDE, out=HALF)), (norm_fp8, dict(x=HALF, stream=WIDE, w=FLOAT, h=WIDE)),
         (backward, dict(h=WIDE, w=FLOAT, dout=HALF, dh=WIDE, dx=HALF, dresidual=WIDE, dw=FLOAT)), (quantise, dict(x=WIDE)),
         (quantise_weight, dict(w=WIDE)), (clip, dict(norm=FLOAT)), (linear, dict(out=WIDE)), (linear_quantise, dict(x=WIDE, out=WIDE))]


@pytest.mark.parametrize("f32", [0, 1])
@pytest.mark.parametrize("call,names", CALLS, ids=lambda v: getattr(v, "__name__", ""))
def test_addresses_off_their_boundary_are_refused(lib, call, names, f32):
    for name, kind in names.items():
        size = 4 if kind == FLOAT or (kind == WIDE and f32) else 2
        for off in range(1, size):
            assert call(lib, f32, **{name: A + off}) == INVALID, (name, off)
