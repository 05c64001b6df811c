"""Which output belongs to which gradient, where either comes as a dict.  No GPU: the addresses that reach the library."""
import ctypes

import pytest
import torch

import matrix_state_nonlinear_gb300 as pkg
from matrix_state_nonlinear_gb300 import layer
from test_layer_binding import BF16, F32
from test_ssm_binding import Fake


class At(Fake):
    def __init__(self, at, *shape, dtype=F32):
        super().__init__(0, *shape, dtype=dtype)
        self.at = at

    def data_ptr(self):
        return self.at


@pytest.fixture
def pairs(monkeypatch):
    """The (input, output) addresses of the last clip."""
    found = []

    class Library:
        def m2rnn_grad_norm_workspace_bytes(self, n):
            return 64

        def m2rnn_clip_grad_norm(self, grads, out, values, kinds, n, *rest):
            read = lambda p: (ctypes.c_uint64 * n).from_address(p)[:]  # noqa: E731
            found[:] = zip(read(grads), read(out))
            return layer.OK

    monkeypatch.setattr(layer, "load_library", Library)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    return found


def run(grads, out):
    return pkg.clip_grad_norm(grads, 1.0, out=out, norm=At(64, dtype=F32), workspace=At(128, 64, dtype=torch.uint8))


def test_dicts_are_matched_by_name(pairs):
    grads = {"a": At(1000, 4), "b": At(2000, 4), "c": At(3000, 4)}
    run(grads, {"c": At(6000, 4), "a": At(4000, 4), "b": At(5000, 4)})
    assert pairs == [(1000, 4000), (2000, 5000), (3000, 6000)]
    run(grads, [At(4000, 4), At(5000, 4), At(6000, 4)])
    assert pairs == [(1000, 4000), (2000, 5000), (3000, 6000)]
    run(grads, None)
    assert pairs == [(n, n) for n in (1000, 2000, 3000)]


def test_other_names_are_refused(pairs):
    grads = {"a": At(1000, 4), "b": At(2000, 4)}
    for out in ({"a": At(4000, 4), "c": At(5000, 4)}, {"a": At(4000, 4)}, {"a": At(4000, 4), "b": At(5000, 4), "c": At(6000, 4)}):
        with pytest.raises(ValueError, match="out"):
            run(grads, out)
    with pytest.raises(TypeError):
        run(grads, {"a": At(4000, 4), "b": At(5000, 4, dtype=BF16)})
    assert not pairs
