"""What the binding of the residual norm, the 8-bit values and the clip refuses before any launch, without a GPU:
stand-ins for tensors as in the selective block's test, and the C entries on addresses that are never read."""
import ctypes
from array import array

import pytest
import torch

import __graft_entry__
import matrix_state_nonlinear_gb300 as pkg
from matrix_state_nonlinear_gb300 import layer
from matrix_state_nonlinear_gb300 import m2rnn as binding
from test_ssm_binding import Fake

BF16, F32, FP8, E8M0 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu


class Reached(Exception):
    pass


class Stub:
    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                return 64
            raise Reached(name)
        return call


@pytest.fixture
def stub(monkeypatch):
    monkeypatch.setattr(layer, "load_library", Stub)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)


def parts(dev, M=6, K=256, N=128):
    t = lambda *s, dtype=BF16: Fake(dev, *s, dtype=dtype)  # noqa: E731
    return dict(x=t(M, K), r=t(M, K, dtype=F32), w=t(K, dtype=F32), out=t(M, K), h=t(M, K, dtype=F32), q=t(M, K, dtype=FP8),
                s=t(M, K // 128, dtype=E8M0), wt=t(N, K), wq=t(N, K, dtype=FP8), ws=t(N // 128, K // 128, dtype=E8M0),
                y=t(M, N), space=t(4096, dtype=torch.uint8), dw=t(K, dtype=F32), norm=t(dtype=F32))


CALLS = {
    "add_rmsnorm": lambda p: pkg.add_rmsnorm(p["x"], p["r"], p["w"], out=p["out"], h=p["h"]),
    "add_rmsnorm_fp8": lambda p: pkg.add_rmsnorm_fp8(p["x"], p["r"], p["w"], out=p["q"], scales=p["s"], h=p["h"]),
    "add_rmsnorm_backward": lambda p: pkg.add_rmsnorm_backward(p["h"], p["w"], p["out"], p["r"], grads=dict(dx=p["x"], dresidual=p["r"], dw=p["dw"]),
                                                               workspace=p["space"]),
    "quantise_fp8": lambda p: pkg.quantise_fp8(p["x"], p["q"], p["s"]),
    "quantise_weight_fp8": lambda p: pkg.quantise_weight_fp8(p["wt"], p["wq"], p["ws"]),
    "linear_fp8": lambda p: pkg.linear_fp8(p["q"], p["s"], p["wq"], p["ws"], out=p["y"]),
    "linear_fp8 of bf16": lambda p: pkg.linear_fp8(p["x"], None, p["wq"], p["ws"], out=p["y"], workspace=p["space"]),
    "clip_grad_norm": lambda p: pkg.clip_grad_norm([p["x"], p["r"]], 1.0, norm=p["norm"], workspace=p["space"]),
    "grad_norm": lambda p: pkg.grad_norm([p["x"], p["r"]], norm=p["norm"], workspace=p["space"]),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_another_device_is_refused(stub, name):
    with pytest.raises(Reached):
        CALLS[name](parts(0))
    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
        CALLS[name](parts(1))


@pytest.mark.parametrize("name,which,error", [
    ("add_rmsnorm", dict(w=Fake(0, 255, dtype=F32)), ValueError), ("add_rmsnorm", dict(x=Fake(0, 6, 256, dtype=torch.float16)), TypeError),
    ("add_rmsnorm", dict(r=Fake(0, 6, 256, dtype=torch.float64)), TypeError), ("add_rmsnorm", dict(h=Fake(0, 6, 256)), TypeError),
    ("add_rmsnorm", dict(out=Fake(0, 5, 256)), ValueError), ("add_rmsnorm", dict(w=Fake(1, 256, dtype=F32)), ValueError),
    ("add_rmsnorm_fp8", dict(q=Fake(0, 6, 256, dtype=torch.uint8)), TypeError), ("add_rmsnorm_fp8", dict(s=Fake(0, 6, 3, dtype=E8M0)), ValueError),
    ("add_rmsnorm_fp8", dict(s=Fake(0, 6, 2, dtype=F32)), TypeError), ("add_rmsnorm_backward", dict(out=Fake(0, 6, 255)), ValueError),
    ("quantise_fp8", dict(x=Fake(0, 6, 256, dtype=torch.float16)), TypeError), ("quantise_weight_fp8", dict(ws=Fake(0, 2, 1, dtype=E8M0)), ValueError),
    ("linear_fp8", dict(ws=Fake(0, 1, 2, dtype=F32)), TypeError), ("linear_fp8", dict(wq=Fake(0, 128, 255, dtype=FP8)), ValueError),
    ("linear_fp8", dict(y=Fake(0, 6, 127)), ValueError), ("linear_fp8", dict(y=Fake(0, 6, 128, dtype=torch.float16)), TypeError),
    ("linear_fp8 of bf16", dict(x=Fake(0, 6, 256, dtype=torch.float16)), TypeError),
    ("clip_grad_norm", dict(r=Fake(0, 6, 256, dtype=torch.float16)), TypeError), ("clip_grad_norm", dict(r=Fake(1, 6, 256, dtype=F32)), ValueError),
])
def test_types_shapes_and_devices_are_refused(stub, name, which, error):
    with pytest.raises(error):
        CALLS[name](dict(parts(0), **which))


class Strided(Fake):
    """Rows `row` values apart."""

    def __init__(self, *shape, row, at=1 << 20, dtype=FP8):
        super().__init__(0, *shape, dtype=dtype)
        self.row, self.at = row, at

    def is_contiguous(self):
        return False

    def stride(self, i=None):
        s = (self.row, 1)
        return s if i is None else s[i]

    def data_ptr(self):
        return self.at


def test_8_bit_rows_off_their_boundaries_are_refused(stub):
    with pytest.raises(Reached):
        CALLS["linear_fp8"](dict(parts(0), q=Strided(6, 256, row=272)))
    for q in (Strided(6, 256, row=264), Strided(6, 256, row=272, at=(1 << 20) + 8)):
        with pytest.raises(ValueError, match="16-byte boundaries"):
            CALLS["linear_fp8"](dict(parts(0), q=q))


def test_rows_that_lie_unevenly_are_refused():
    t = torch.zeros(4, 6, 8, dtype=BF16)
    assert layer._rows(t[:, :3].transpose(0, 1)[:, :1], "x", BF16, torch.Size((3, 1, 8)), -1)[1] == 8
    with pytest.raises(ValueError, match="one stride apart"):
        layer._rows(t[:, :3], "x", BF16, torch.Size((4, 3, 8)), -1)
    with pytest.raises(ValueError, match="contiguous"):
        layer._rows(t.transpose(1, 2), "x", BF16, torch.Size((4, 8, 6)), -1)
    assert layer._rows(t[:, :, :5], "x", BF16, torch.Size((4, 6, 5)), -1)[1] == 8


def test_gradient_lists_are_refused(stub):
    p = parts(0)
    with pytest.raises(ValueError):
        pkg.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError):
        pkg.clip_grad_norm([p["x"], p["r"]], 1.0, out=[p["x"]], norm=p["norm"], workspace=p["space"])
    with pytest.raises(TypeError):
        pkg.clip_grad_norm([p["x"]], 1.0, out=[p["r"]], norm=p["norm"], workspace=p["space"])


# ---------------------------------------------------------------- the C entries
@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return binding.load_library()


A = 1 << 20  # an aligned address that is never read
INVALID, UNSUPPORTED, OK = binding.ERR_INVALID_ARG, binding.ERR_UNSUPPORTED, binding.OK


def test_norm_sizes(lib):
    call = lambda rows, D, x=A, h=A, eps=1e-5, out=A: lib.m2rnn_add_rmsnorm(x, D, A, 0, D, A, eps, h, out, rows, D, None)  # noqa: E731
    assert call(-1, 8) == call(4, 0) == call(4, 8, eps=-1.0) == call(4, 8, eps=float("nan")) == INVALID
    assert call(4, 8, h=None) == call(4, 8, out=None) == INVALID
    assert call(4, 16385) == UNSUPPORTED and call(0, 8) == OK
    back = lambda dx, dr, ws, n: lib.m2rnn_add_rmsnorm_backward(A, 0, A, 1e-5, A, None, dx, dr, A, 4, 8, ws, n, None)  # noqa: E731
    need = lib.m2rnn_add_rmsnorm_backward_workspace_bytes(4, 8)
    assert need > 0 and lib.m2rnn_add_rmsnorm_backward_workspace_bytes(4, 16385) == 0
    assert back(None, None, A, need) == back(A, None, None, need) == back(A, None, A + 4, need) == back(A, None, A, need - 1) == INVALID


def test_8_bit_sizes(lib):
    q = lambda rows, D, to=A, row=None: lib.m2rnn_quantise_fp8(A, 0, D, to, (D + 15) // 16 * 16 if row is None else row, A, rows, D, None)  # noqa: E731
    assert q(-1, 8) == q(4, 0) == q(4, 8, to=A + 8) == q(4, 8, row=24) == q(4, 32, row=16) == INVALID and q(0, 8) == OK
    assert q(1 << 40, 8) == UNSUPPORTED
    f = lambda M, N, K, x=A, row=None, w=A: lib.m2rnn_linear_fp8(x, (K + 15) // 16 * 16 if row is None else row, A, w, (K + 15) // 16 * 16, A, A, 0, M, N, K, None)  # noqa: E731
    assert f(-1, 8, 8) == f(4, 0, 8) == f(4, 8, 0) == f(4, 8, 8, x=A + 1) == f(4, 8, 8, row=8) == f(4, 8, 8, w=None) == INVALID
    assert f(0, 8, 8) == OK and f(1 << 31, 8, 8) == f(1 << 30, 1 << 30, 8) == UNSUPPORTED
    assert lib.m2rnn_linear_quantise_workspace_bytes(0, 16, 4096) == 0
    need = lib.m2rnn_linear_quantise_workspace_bytes(1, 16, 1000)
    assert need >= 16 * (1000 + 8)
    g = lambda ws, n: lib.m2rnn_linear_quantise_fp8(A, 1, 1000, A, 1008, A, A, 0, 16, 8, 1000, ws, n, None)  # noqa: E731
    assert g(A, need - 1) == g(None, need) == g(A + 8, need) == INVALID


def clip(lib, ranges, out=None, most=1.0, kinds=None, ws=A, n=None):
    """ranges: (address, values) of each gradient; out: addresses."""
    k = len(ranges)
    p, v = array("Q", [a for a, _ in ranges]), array("q", [n for _, n in ranges])
    t, o = array("B", kinds or [1] * k), array("Q", out if out is not None else [a for a, _ in ranges])
    need = lib.m2rnn_grad_norm_workspace_bytes(k) if n is None else n
    return lib.m2rnn_clip_grad_norm(p.buffer_info()[0], o.buffer_info()[0], v.buffer_info()[0], t.buffer_info()[0], k, most, A, ws, need,
                                    None)


def test_clip_refusals(lib):
    assert clip(lib, [(A, -1)]) == clip(lib, [(0, 4)]) == clip(lib, [(A + 2, 4)]) == clip(lib, [(A + 1, 4)], kinds=[0]) == INVALID
    assert clip(lib, [(A, 4)], most=-1.0) == clip(lib, [(A, 4)], most=float("inf")) == clip(lib, [(A, 4)], most=float("nan")) == INVALID
    assert clip(lib, [(A, 4)], ws=None) == clip(lib, [(A, 4)], ws=A + 8) == clip(lib, [(A, 4)], n=8) == INVALID
    assert clip(lib, [(A, 1 << 41)]) == clip(lib, [(A, 1 << 39)] * 3) == UNSUPPORTED
    # shared memory: the same twice, overlaps, an output on another's input
    assert clip(lib, [(A, 4), (A, 4)]) == clip(lib, [(A, 8), (A + 16, 8)]) == INVALID
    assert clip(lib, [(A, 8), (A + 4096, 8)], out=[A + 4096, A + 8192]) == clip(lib, [(A, 8)], out=[A + 4]) == INVALID
    assert clip(lib, [(A, 64), (A + 4096, 8)], out=[A + 8192, A + 8192 + 128]) == INVALID
    assert lib.m2rnn_clip_grad_norm(None, None, None, None, 1, 1.0, ctypes.c_void_p(A), A, 1 << 20, None) == INVALID
