"""The scan after its CUDA context is replaced, and in a second context of one process.

Function attributes and symbol addresses belong to a context (or go with it).  Child processes run
forward and backward through the C entries in one context, then in another, and compare the bits.
"""
import os
import subprocess
import sys

import pytest
import torch

import __graft_entry__

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import ctypes, sys
import torch
import matrix_state_nonlinear_gb300 as pkg

how, (B, T, N, G, K, V) = sys.argv[1], (int(x) for x in sys.argv[2:])
cu = ctypes.CDLL("libcuda.so.1")
P, S, I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
cu.cuCtxCreate_v2.argtypes = [ctypes.POINTER(P), ctypes.c_uint, I]
cu.cuDevicePrimaryCtxRetain.argtypes = [ctypes.POINTER(P), I]
cu.cuDevicePrimaryCtxReset_v2.argtypes = [I]
cu.cuCtxSetCurrent.argtypes = [P]
cu.cuMemAlloc_v2.argtypes = [ctypes.POINTER(P), S]
cu.cuMemcpyHtoD_v2.argtypes = [P, P, S]
cu.cuMemcpyDtoH_v2.argtypes = [P, P, S]

def ok(r, what):
    if r != 0:
        sys.exit(f"{what}: error {r}")

gen = torch.Generator().manual_seed(0)
bf = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16)
s = dict(q=bf(B, T, G, K), k=bf(B, T, G, K), v=bf(B, T, N, V), a=bf(B, T, N), alpha=torch.rand(N, generator=gen) + 0.1,
         beta=torch.randn(N, generator=gen), w_r=torch.randn(N, V, generator=gen))
dy = bf(B, T, N, V)
names = ("y", "H_T", "dq", "dk", "dv", "da", "dalpha", "dbeta", "dw_r", "dH0")
outs = [torch.empty(z, dtype=t) for z, t in zip(
    [(B, T, N, V), (B, N, K, V), (B, T, G, K), (B, T, G, K), (B, T, N, V), (B, T, N), (N,), (N,), (N, V), (B, N, K, V)],
    [torch.bfloat16, torch.float32] + 4 * [torch.bfloat16] + 4 * [torch.float32])]
lib = pkg.load_library()

def alloc(nbytes):
    p = P()
    ok(cu.cuMemAlloc_v2(ctypes.byref(p), max(nbytes, 256)), "memory")
    return p.value

def size(t):
    return t.numel() * t.element_size()

def put(t):
    p = alloc(size(t))
    ok(cu.cuMemcpyHtoD_v2(p, t.data_ptr(), size(t)), "copy in")
    return p

def run():
    # Forward and backward in the current context: the outputs on the host.
    ins = [put(t) for t in s.values()]
    out = [alloc(size(t)) for t in outs]
    hs = alloc(lib.m2rnn_ssm_states_bytes(B, T, N, K, V))
    fb, bb = (lib.m2rnn_ssm_workspace_bytes(B, T, N, G, K, V, i) for i in (0, 1))
    ok(lib.m2rnn_ssm_forward_bf16(*ins, None, *out[:2], hs, None, B, T, N, G, K, V, alloc(fb), fb, None), "forward")
    ok(lib.m2rnn_ssm_backward_bf16(*ins, hs, put(dy), None, *out[2:], None, B, T, N, G, K, V, alloc(bb), bb, None),
       "backward")
    ok(lib.m2rnn_stream_status(None), "status")
    got = [torch.empty_like(t) for t in outs]
    for t, p in zip(got, out):
        ok(cu.cuMemcpyDtoH_v2(t.data_ptr(), p, size(t)), "copy out")
    return got

ctx = P()
ok(cu.cuInit(0), "init")
ok(cu.cuDevicePrimaryCtxRetain(ctypes.byref(ctx), 0), "context")
ok(cu.cuCtxSetCurrent(ctx), "context")
want = run()
if how == "replaced":  # this process's own context ends, a new one takes its place
    ok(cu.cuDevicePrimaryCtxReset_v2(0), "reset")
    ok(cu.cuDevicePrimaryCtxRetain(ctypes.byref(ctx), 0), "context")
    ok(cu.cuCtxSetCurrent(ctx), "context")
else:
    ok(cu.cuCtxCreate_v2(ctypes.byref(ctx), 0, 0), "context")  # and current from here on
for n, a, b in zip(names, run(), want):
    if not torch.equal(a, b):
        sys.exit(f"{n} differs in the other context")
print("the same bits")
"""


# K on both sides of 64; a sequence cut into segments (the states' kernels in both forms).
@pytest.mark.parametrize("shape", [(2, 200, 2, 1, 64, 64), (1, 1100, 2, 1, 128, 64)])
@pytest.mark.parametrize("how", ["second", "replaced"])
def test_scan_in_another_context(how, shape):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    __graft_entry__.build()
    r = subprocess.run([sys.executable, "-c", CHILD, how, *map(str, shape)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-500:] + r.stderr[-2000:]
    assert "the same bits" in r.stdout
