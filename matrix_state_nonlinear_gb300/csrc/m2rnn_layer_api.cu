// m2rnn_layer_api.cu — C entries of what stands around a block in a stack (residual RMS norm, 8-bit
// projections, the clipping of gradients): argument checks, then the launchers.  A failed check launches
// nothing; nothing here allocates device memory or waits.
#include <algorithm>
#include <math.h>
#include <memory>
#include <new>

#include "../../include/m2rnn.h"
#include "m2rnn_layer.h"

using namespace m2rnn;

namespace {

m2rnn_status done(cudaError_t e) { return e == cudaSuccess ? M2RNN_OK : M2RNN_ERR_CUDA; }

m2rnn_status row_sizes(long long rows, int D) {
  if (rows < 0 || D < 1) return M2RNN_ERR_INVALID_ARG;
  return D > kNormMaxRow ? M2RNN_ERR_UNSUPPORTED : M2RNN_OK;
}

size_t size_of(int f32) { return f32 ? 4 : 2; }

// Rows of 8-bit values that start on 16-byte boundaries.
bool byte_rows(const void* p, long long row, int width) {
  return aligned_to(p, 16) && row % 16 == 0 && row >= width;
}

// A range of memory of tensor `tensor`; `written` where a call writes it.
struct Range {
  uintptr_t from, to;
  bool written;
};
// Whether a written range shares memory with any other; the ranges are sorted by `from`.
bool written_overlap(const Range* r, size_t n) {
  uintptr_t any = 0, written = 0;  // ends of the ranges so far
  for (size_t i = 0; i < n; ++i) {
    if (r[i].from < (r[i].written ? any : written)) return true;
    any = std::max(any, r[i].to);
    if (r[i].written) written = std::max(written, r[i].to);
  }
  return false;
}

}  // namespace

extern "C" {

static m2rnn_status add_norm_problem(const uint16_t* x, long long x_row, const void* stream_in, int stream_f32,
                                     long long stream_row, const float* w, float eps, void* h, long long rows, int D,
                                     AddNormProblem* p) {
  const m2rnn_status st = row_sizes(rows, D);
  if (st != M2RNN_OK) return st;
  if (!(eps >= 0.f) || !w || x_row < 0 || stream_row < 0) return M2RNN_ERR_INVALID_ARG;
  if (rows > 0 && (!stream_in || (x && !h))) return M2RNN_ERR_INVALID_ARG;
  const size_t size = size_of(stream_f32);
  if (!aligned_to(x, 2) || !aligned_to(stream_in, size) || !aligned_to(w, 4) || !aligned_to(h, size))
    return M2RNN_ERR_INVALID_ARG;
  *p = AddNormProblem{x, stream_in, x_row, stream_row, stream_f32 != 0, w, eps, h, rows, D};
  return M2RNN_OK;
}

m2rnn_status m2rnn_add_rmsnorm(const uint16_t* x, long long x_row, const void* stream_in, int stream_f32,
                               long long stream_row, const float* w, float eps, void* h, uint16_t* out, long long rows,
                               int D, void* stream) {
  AddNormProblem p;
  const m2rnn_status st = add_norm_problem(x, x_row, stream_in, stream_f32, stream_row, w, eps, h, rows, D, &p);
  if (st != M2RNN_OK || rows == 0) return st;
  if (!out || !aligned_to(out, 2)) return M2RNN_ERR_INVALID_ARG;
  return done(launch_add_rmsnorm(p, out, static_cast<cudaStream_t>(stream)));
}

m2rnn_status m2rnn_add_rmsnorm_fp8(const uint16_t* x, long long x_row, const void* stream_in, int stream_f32,
                                   long long stream_row, const float* w, float eps, void* h, uint8_t* q,
                                   long long q_row, uint8_t* scales, long long rows, int D, void* stream) {
  AddNormProblem p;
  const m2rnn_status st = add_norm_problem(x, x_row, stream_in, stream_f32, stream_row, w, eps, h, rows, D, &p);
  if (st != M2RNN_OK || rows == 0) return st;
  if (!q || !scales || !byte_rows(q, q_row, D)) return M2RNN_ERR_INVALID_ARG;
  return done(launch_add_rmsnorm_fp8(p, q, q_row, scales, static_cast<cudaStream_t>(stream)));
}

size_t m2rnn_add_rmsnorm_backward_workspace_bytes(long long rows, int D) {
  return row_sizes(rows, D) == M2RNN_OK ? sizeof(float) * add_rmsnorm_backward_workspace_floats(rows, D) : 0;
}

m2rnn_status m2rnn_add_rmsnorm_backward(const void* h, int stream_f32, const float* w, float eps, const uint16_t* dout,
                                        const void* dh, uint16_t* dx, void* dresidual, float* dw, long long rows, int D,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  const m2rnn_status st = row_sizes(rows, D);
  if (st != M2RNN_OK) return st;
  if (!(eps >= 0.f) || !w || !dw) return M2RNN_ERR_INVALID_ARG;
  if (rows > 0 && (!h || !dout || !workspace || (!dx && !dresidual))) return M2RNN_ERR_INVALID_ARG;
  if (!aligned_to(workspace, 16) || workspace_bytes < m2rnn_add_rmsnorm_backward_workspace_bytes(rows, D))
    return M2RNN_ERR_INVALID_ARG;
  const size_t size = size_of(stream_f32);
  if (!aligned_to(h, size) || !aligned_to(w, 4) || !aligned_to(dout, 2) || !aligned_to(dh, size) || !aligned_to(dx, 2) ||
      !aligned_to(dresidual, size) || !aligned_to(dw, 4))
    return M2RNN_ERR_INVALID_ARG;
  const AddNormBackwardProblem p{h,  stream_f32 != 0, w, eps, dout, dh, dx, dresidual, dw, rows,
                                 D,  static_cast<float*>(workspace)};
  return done(launch_add_rmsnorm_backward(p, static_cast<cudaStream_t>(stream)));
}

m2rnn_status m2rnn_quantise_fp8(const void* x, int x_f32, long long x_row, uint8_t* q, long long q_row, uint8_t* scales,
                                long long rows, int D, void* stream) {
  if (rows < 0 || D < 1 || x_row < 0) return M2RNN_ERR_INVALID_ARG;
  if ((rows + 1) > 0x7ffffff0LL * 16 / scale_blocks(D)) return M2RNN_ERR_UNSUPPORTED;
  if (rows == 0) return M2RNN_OK;
  if (!x || !aligned_to(x, size_of(x_f32)) || !q || !scales || !byte_rows(q, q_row, D)) return M2RNN_ERR_INVALID_ARG;
  return done(launch_quantise_rows(x, x_f32 != 0, x_row, q, q_row, scales, rows, D, static_cast<cudaStream_t>(stream)));
}

m2rnn_status m2rnn_quantise_weight_fp8(const void* w, int w_f32, long long w_row, uint8_t* q, long long q_row,
                                       uint8_t* scales, int N, int K, void* stream) {
  if (N < 1 || K < 1 || w_row < 0) return M2RNN_ERR_INVALID_ARG;
  if ((long long)scale_blocks(N) * scale_blocks(K) > 0x7fffffffLL) return M2RNN_ERR_UNSUPPORTED;
  if (!w || !aligned_to(w, size_of(w_f32)) || !q || !scales || !byte_rows(q, q_row, K)) return M2RNN_ERR_INVALID_ARG;
  return done(launch_quantise_weight(w, w_f32 != 0, w_row, q, q_row, scales, N, K, static_cast<cudaStream_t>(stream)));
}

// Sizes of a product and its weights.  Rows are tensor-map coordinates and the tiles, of 128 x 16 at the
// least, a grid, both in 31 bits; a tensor map's stride has 40.
static m2rnn_status linear_checks(const uint8_t* w, long long w_row, const uint8_t* w_scales, const void* out,
                                  int out_f32, long long M, int N, int K) {
  if (M < 0 || N < 1 || K < 1) return M2RNN_ERR_INVALID_ARG;
  if (M > 0x7fffff00LL || N > 0x7fffff00 || K > 0x7fffff00 || ((M + 15) / 16) * ((N + 127LL) / 128) > 0x7fffffffLL)
    return M2RNN_ERR_UNSUPPORTED;
  if (M == 0) return M2RNN_OK;
  if (!w || !w_scales || !out || !aligned_to(out, size_of(out_f32)) || !byte_rows(w, w_row, K))
    return M2RNN_ERR_INVALID_ARG;
  return w_row >= 1LL << 40 ? M2RNN_ERR_UNSUPPORTED : M2RNN_OK;
}

m2rnn_status m2rnn_linear_fp8(const uint8_t* x, long long x_row, const uint8_t* x_scales, const uint8_t* w,
                              long long w_row, const uint8_t* w_scales, void* out, int out_f32, long long M, int N,
                              int K, void* stream) {
  const m2rnn_status st = linear_checks(w, w_row, w_scales, out, out_f32, M, N, K);
  if (st != M2RNN_OK || M == 0) return st;
  if (!x || !x_scales || !byte_rows(x, x_row, K)) return M2RNN_ERR_INVALID_ARG;
  if (x_row >= 1LL << 40) return M2RNN_ERR_UNSUPPORTED;
  int* status = device_status();
  if (!status) return M2RNN_ERR_CUDA;
  const LinearProblem p{x, x_scales, nullptr, w, w_scales, x_row, w_row, out, out_f32 != 0, (int)M, N, K, status};
  return done(launch_linear_fp8(p, static_cast<cudaStream_t>(stream)));
}

// Bytes from row to row of activations in the workspace: rows start on lines of the cache, short ones on 16 bytes.
static long long quantised_row(int K) { return K > 128 ? (K + 127LL) / 128 * 128 : (K + 15LL) / 16 * 16; }

size_t m2rnn_linear_quantise_workspace_bytes(int x_f32, long long M, int K) {
  if (M < 1 || M > 0x7fffff00LL || K < 1 || (M <= kRawRows && !x_f32)) return 0;
  return (size_t)M * (quantised_row(K) + scale_blocks(K));  // q, then its scales
}

m2rnn_status m2rnn_linear_quantise_fp8(const void* x, int x_f32, long long x_row, const uint8_t* w, long long w_row,
                                       const uint8_t* w_scales, void* out, int out_f32, long long M, int N, int K,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  m2rnn_status st = linear_checks(w, w_row, w_scales, out, out_f32, M, N, K);
  if (st != M2RNN_OK || M == 0) return st;
  if (!x || x_row < 0 || !aligned_to(x, size_of(x_f32))) return M2RNN_ERR_INVALID_ARG;
  const size_t need = m2rnn_linear_quantise_workspace_bytes(x_f32, M, K);
  if (need > 0 && (!workspace || !aligned_to(workspace, 16) || workspace_bytes < need)) return M2RNN_ERR_INVALID_ARG;
  int* status = device_status();
  if (!status) return M2RNN_ERR_CUDA;
  const auto at = static_cast<cudaStream_t>(stream);
  LinearProblem p{nullptr, nullptr, nullptr, w, w_scales, x_row, w_row, out, out_f32 != 0, (int)M, N, K, status};
  if (need > 0) {
    p.x_row = quantised_row(K);
    uint8_t *q = static_cast<uint8_t*>(workspace), *scales = q + M * p.x_row;
    st = done(launch_quantise_rows(x, x_f32 != 0, x_row, q, p.x_row, scales, M, K, at));
    if (st != M2RNN_OK) return st;
    p.x = q, p.x_scales = scales, p.follows = true;
  } else {
    p.raw = static_cast<const uint16_t*>(x);
  }
  return done(launch_linear_fp8(p, at));
}

size_t m2rnn_grad_norm_workspace_bytes(int count) { return count >= 0 ? grad_norm_workspace_bytes(count) : 0; }

m2rnn_status m2rnn_clip_grad_norm(const void* const* grads, void* const* out, const long long* values,
                                  const unsigned char* is_f32, int count, float max_norm, float* norm, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (count < 0 || !norm || !aligned_to(norm, 4)) return M2RNN_ERR_INVALID_ARG;
  if (out && !(max_norm >= 0.f && max_norm <= 3.402823466e38f)) return M2RNN_ERR_INVALID_ARG;
  if (count > 0 && (!grads || !values || !is_f32 || !workspace || !aligned_to(workspace, 16) ||
                    workspace_bytes < m2rnn_grad_norm_workspace_bytes(count)))
    return M2RNN_ERR_INVALID_ARG;
  long long total = 0;
  for (int i = 0; i < count; ++i) {
    const size_t size = size_of(is_f32[i]);
    if (values[i] < 0 || (values[i] > 0 && (!grads[i] || (out && !out[i])))) return M2RNN_ERR_INVALID_ARG;
    if (values[i] > 0 && (!aligned_to(grads[i], size) || (out && !aligned_to(out[i], size))))
      return M2RNN_ERR_INVALID_ARG;
    if (values[i] > kMaxGradValues - total) return M2RNN_ERR_UNSUPPORTED;
    total += values[i];
  }
  if (out && count > 0) {
    const std::unique_ptr<Range[]> r(new (std::nothrow) Range[2 * (size_t)count]);
    if (!r) return M2RNN_ERR_CUDA;
    size_t n = 0;
    for (int i = 0; i < count; ++i) {
      const uintptr_t bytes = (uintptr_t)values[i] * (is_f32[i] ? 4 : 2), a = reinterpret_cast<uintptr_t>(grads[i]),
                      b = reinterpret_cast<uintptr_t>(out[i]);
      if (bytes == 0) continue;
      r[n++] = Range{b, b + bytes, true};
      if (a != b) r[n++] = Range{a, a + bytes, false};
    }
    const auto before = [](const Range& x, const Range& y) { return x.from < y.from; };
    if (!std::is_sorted(r.get(), r.get() + n, before)) std::sort(r.get(), r.get() + n, before);
    if (written_overlap(r.get(), n)) return M2RNN_ERR_INVALID_ARG;
  }
  const GradProblem p{grads, out, values, is_f32, count, max_norm, norm, workspace};
  return done(launch_grad_norm(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
