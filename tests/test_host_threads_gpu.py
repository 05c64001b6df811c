"""Calls from several host threads, each on a stream of its own and each of another size, so that they meet in one
kernel with different blocks: every launch is accepted and gives the bits of a call alone.  A program on the C
entries calls as often as a host can, without Python's lock between the calls."""
import os
import subprocess
import threading

import pytest
import torch

import matrix_state_nonlinear_gb300 as pkg
from matrix_state_nonlinear_gb300 import build
from test_layer_gpu import BF16, DEV, F32, built, rand  # noqa: F401

pytestmark = pytest.mark.gpu


def at_once(calls, times):
    """Each of `calls` (name -> function of a stream that returns tensors) in a thread of its own, `times` times."""
    want = {n: [t.clone() for t in f(torch.cuda.current_stream())] for n, f in calls.items()}
    torch.cuda.synchronize()
    start, errors, got = threading.Barrier(len(calls)), [], {}

    def run(name, f):
        try:
            torch.cuda.set_device(DEV)
            stream = torch.cuda.Stream()
            start.wait(60)
            for _ in range(times):
                out = f(stream)
            stream.synchronize()
            got[name] = out
        except Exception as e:  # reported by the test's own thread
            errors.append((name, repr(e)))

    threads = [threading.Thread(target=run, args=item) for item in calls.items()]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not errors and not any(t.is_alive() for t in threads), errors
    for n, w in want.items():
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got[n], w)), n
    assert pkg.stream_status() == 0


def bits(t):
    return t.view(torch.uint8) if t.dtype.itemsize == 1 else t


def backward(D, dtype):
    h, w, dout = rand((16, D), D, 1.0, dtype), rand((D,), D + 1, 1.0, F32), rand((16, D), D + 2)
    grads = dict(dx=torch.empty_like(dout), dresidual=torch.empty_like(h), dw=torch.empty_like(w))
    space = torch.empty(pkg.load_library().m2rnn_add_rmsnorm_backward_workspace_bytes(16, D), dtype=torch.uint8, device=DEV)
    return lambda stream: list(pkg.add_rmsnorm_backward(h, w, dout, None, grads=grads, workspace=space, stream=stream).values())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("sizes", [(2048, 4096, 1024), (2047, 4095, 1023), (4104, 8192, 6000), (16384, 12000, 9001)])
def test_norm_backward(sizes, dtype):
    at_once({D: backward(D, dtype) for D in sizes}, 300)


def eight(D, dtype):
    r, w = rand((16, D), D, 1.0, dtype), rand((D,), D + 1, 1.0, F32)
    first = pkg.add_rmsnorm_fp8(r, None, w)[:2]
    out = dict(zip(("out", "scales"), first))
    return lambda stream: list(pkg.add_rmsnorm_fp8(r, None, w, **out, stream=stream)[:2])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_in_8_bits(dtype):
    at_once({D: eight(D, dtype) for D in (9001, 16001, 12345)}, 300)


PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <thread>
#include <vector>
#include <cuda_runtime.h>
#include "m2rnn.h"
static char* room(size_t n) {  // zeros, which every call takes
  void* p = nullptr;
  if (cudaMalloc(&p, n) != cudaSuccess || cudaMemset(p, 0, n) != cudaSuccess) std::exit(2);
  return static_cast<char*>(p);
}
using Call = std::function<m2rnn_status(cudaStream_t)>;
static Call norm_backward(int f32, int D) {
  const size_t ws = m2rnn_add_rmsnorm_backward_workspace_bytes(4, D);
  char *t = room(4 << 20), *s = room(ws);
  const uint16_t* dout = reinterpret_cast<uint16_t*>(t + (1 << 20));
  uint16_t* dx = reinterpret_cast<uint16_t*>(t + (2 << 20));
  float *w = reinterpret_cast<float*>(t + (3 << 20)), *dw = w + 65536;
  return [=](cudaStream_t at) { return m2rnn_add_rmsnorm_backward(t, f32, w, 1e-5f, dout, nullptr, dx, nullptr, dw, 4, D, s, ws, at); };
}
static Call norm_fp8(int f32, int D) {
  char* t = room(4 << 20);
  uint8_t *q = reinterpret_cast<uint8_t*>(t + (1 << 20)), *scales = q + (1 << 20);
  float* w = reinterpret_cast<float*>(t + (3 << 20));
  return [=](cudaStream_t at) { return m2rnn_add_rmsnorm_fp8(nullptr, 0, t, f32, D, w, 1e-5f, nullptr, q, (D + 15) / 16 * 16, scales, 4, D, at); };
}
// The recurrence, one step for one head: n is K, or K and V.
static Call forward_f32(int n) {
  float *t = reinterpret_cast<float*>(room(4 << 20)), *y = reinterpret_cast<float*>(room(1 << 20));
  return [=](cudaStream_t at) { return m2rnn_forward_f32(t, t, t, t, t, t, t, t, nullptr, y, nullptr, 1, 1, 1, n, n, at); };
}
static Call backward_f32(int n) {
  const size_t ws = m2rnn_backward_workspace_bytes(1, 1, 1, 1, n, n);
  float *t = reinterpret_cast<float*>(room(4 << 20)), *g = reinterpret_cast<float*>(room(1 << 20));
  char* s = room(ws);
  return [=](cudaStream_t at) {
    float* o[9];
    for (int i = 0; i < 9; ++i) o[i] = g + i * 16384;
    return m2rnn_backward_f32(t, t, t, t, t, t, t, t, nullptr, t, t, nullptr, o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7], nullptr,
                              1, 1, 1, 1, n, n, s, ws, at);
  };
}
static Call forward_bf16(int variant, int V, int n) {
  char *t = room(4 << 20), *y = room(1 << 20);
  const uint16_t* u = reinterpret_cast<uint16_t*>(t);
  const float* f = reinterpret_cast<float*>(t);
  float* o = reinterpret_cast<float*>(y);
  return [=](cudaStream_t at) {
    return m2rnn_forward_bf16_variant(u, u, u, u, f, f, u, f, nullptr, o, nullptr, 1, 8, 1, n, V, variant, at);
  };
}
int main(int argc, char** argv) {
  if (argc < 4) return 2;
  const int times = std::atoi(argv[2]);
  std::vector<Call> calls;
  for (int i = 3; i < argc; ++i) {
    const int n = std::atoi(argv[i]);
    if (!std::strcmp(argv[1], "norm_backward bf16")) calls.push_back(norm_backward(0, n));
    if (!std::strcmp(argv[1], "norm_backward f32")) calls.push_back(norm_backward(1, n));
    if (!std::strcmp(argv[1], "norm_fp8 bf16")) calls.push_back(norm_fp8(0, n));
    if (!std::strcmp(argv[1], "norm_fp8 f32")) calls.push_back(norm_fp8(1, n));
    if (!std::strcmp(argv[1], "forward f32")) calls.push_back(forward_f32(n));
    if (!std::strcmp(argv[1], "backward f32")) calls.push_back(backward_f32(n));
    for (int v = 1; v < 10; ++v)
      if (m2rnn_variant_name(v) && !std::strcmp(argv[1], m2rnn_variant_name(v))) calls.push_back(forward_bf16(v, 64, n));
  }
  std::vector<std::thread> threads;
  std::vector<int> refused(calls.size());
  for (size_t i = 0; i < calls.size(); ++i)
    threads.emplace_back([&, i] {
      cudaStream_t at;
      if (cudaStreamCreateWithFlags(&at, cudaStreamNonBlocking) != cudaSuccess) std::exit(2);
      for (int n = 0; n < times; ++n) {
        refused[i] += calls[i](at) != M2RNN_OK;
        if (n % 256 == 255) cudaStreamSynchronize(at);
      }
      cudaStreamSynchronize(at);
    });
  for (auto& t : threads) t.join();
  int all = 0;
  for (size_t i = 0; i < calls.size(); ++i) {
    std::printf("%s %s: %d of %d calls refused\n", argv[1], argv[3 + i], refused[i], times);
    all += refused[i];
  }
  const int status = m2rnn_stream_status(nullptr);
  if (all || status || cudaDeviceSynchronize() != cudaSuccess) return std::printf("status %d\n", status), 1;
  return calls.empty();
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    at = tmp_path_factory.mktemp("threads")
    src, exe = at / "threads.cpp", at / "threads"
    src.write_text(PROGRAM)
    subprocess.run([build.nvcc(), "-std=c++17", f"-I{build.INCLUDE}", str(src), "-o", str(exe), build.LIB,
                    "-Xlinker", f"-rpath={os.path.dirname(build.LIB)}", "-Xcompiler", "-pthread"], check=True, capture_output=True)
    return str(exe)


@pytest.mark.parametrize("call,sizes", [
    ("norm_backward bf16", (2048, 4096, 1024)), ("norm_backward f32", (2047, 4095, 1023)),
    ("norm_fp8 bf16", (9001, 16001, 12345)), ("norm_fp8 f32", (9001, 16001, 12345)),
    ("forward f32", (128, 96, 16)), ("backward f32", (128, 96, 120)), ("mma_sync_rowwarp", (128, 64, 96)),
    ("mma_sync_pipelined", (64, 48, 32)), ("mma_sync_rows8", (64, 32)),
])
def test_no_launch_is_refused(program, call, sizes):
    r = subprocess.run([program, call, "20000" if call.startswith("norm") else "8000", *map(str, sizes)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
