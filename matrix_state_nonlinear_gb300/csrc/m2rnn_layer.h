// m2rnn_layer.h — what stands around a block in a stack (residual RMS norm, 8-bit projections, the
// clipping of gradients): problem descriptions shared by the C entries (m2rnn_layer_api.cu) and the
// launchers.
//
// 8-bit values are e4m3 with one scale, a power of two kept as its exponent in a byte (e8m0), for each
// 128 consecutive values of a row, the last block of a row being the shorter one.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "m2rnn_ssm.h"

namespace m2rnn {

constexpr int kScaleBlock = 128;  // values that share a scale
// Of n >= 1 values, up to 2^31 - 1 of them.
__host__ __device__ inline int scale_blocks(int n) { return (n - 1) / kScaleBlock + 1; }

constexpr int kNormMaxRow = 16384;  // channels of a row of the norm

struct AddNormProblem {
  const uint16_t* x;     // bf16, or null: h = stream
  const void* stream;    // bf16 or float32 (stream_f32)
  long long x_row, stream_row;  // elements from row to row
  bool stream_f32;
  const float* w;
  float eps;
  void* h;               // of the stream's type, or null
  long long rows;
  int D;
};
cudaError_t launch_add_rmsnorm(const AddNormProblem& p, uint16_t* out, cudaStream_t stream);
cudaError_t launch_add_rmsnorm_fp8(const AddNormProblem& p, uint8_t* q, long long q_row, uint8_t* scales,
                                   cudaStream_t stream);

struct AddNormBackwardProblem {
  const void* h;
  bool stream_f32;
  const float* w;
  float eps;
  const uint16_t* dout;
  const void* dh;   // of the stream's type, or null
  uint16_t* dx;     // or null
  void* dresidual;  // of the stream's type, or null
  float* dw;
  long long rows;
  int D;
  float* ws;
};
size_t add_rmsnorm_backward_workspace_floats(long long rows, int D);
cudaError_t launch_add_rmsnorm_backward(const AddNormBackwardProblem& p, cudaStream_t stream);

// Rows of x (bf16 or float32) to e4m3 in blocks of 128 along a row, and weights in blocks of 128 x 128.
cudaError_t launch_quantise_rows(const void* x, bool f32, long long x_row, uint8_t* q, long long q_row,
                                 uint8_t* scales, long long rows, int D, cudaStream_t stream);
cudaError_t launch_quantise_weight(const void* w, bool f32, long long w_row, uint8_t* q, long long q_row,
                                   uint8_t* scales, int N, int K, cudaStream_t stream);

// Rows of scales, `blocks` bytes each and one behind the other from any address on, are read as whole words of memory.
// The block, of the row at `row`, that the word of block i starts with: i, or up to three less.
__host__ __device__ inline int word_start(const uint8_t* row, int i) {
  return i - (int)(reinterpret_cast<uintptr_t>(row + i) & 3u);
}
// Whether words of row m of `rows` hold bytes outside the tensor.
__host__ __device__ inline bool words_leave(const uint8_t* scales, long long rows, int blocks, long long m) {
  const uintptr_t from = reinterpret_cast<uintptr_t>(scales), row = from + m * blocks;
  return (row & ~(uintptr_t)3) < from || ((row + blocks + 3) & ~(uintptr_t)3) > from + rows * blocks;
}

struct LinearProblem {
  const uint8_t *x, *x_scales;  // [M, K], [M, scale_blocks(K)]
  const uint16_t* raw;          // or, for up to kRawRows tokens, x as bf16, x_row elements from row to row
  const uint8_t *w, *w_scales;  // [N, K], [scale_blocks(N), scale_blocks(K)]
  long long x_row, w_row;       // from row to row; bytes are multiples of 16
  void* out;                    // [M, N] bf16 or float32
  bool out_f32;
  int M, N, K;
  int* status;
  bool follows = false;         // launched behind the quantising of x, which writes nothing else: may start early
};
constexpr int kRawRows = 16;
cudaError_t launch_linear_fp8(const LinearProblem& p, cudaStream_t stream);
cudaError_t launch_linear_pair(const LinearProblem& p, cudaStream_t stream);  // many tokens

// The norm of `count` tensors (with `out`: their scaling to at most max_norm).
struct GradProblem {
  const void* const* in;
  void* const* out;         // in[i] itself or a tensor apart, or null: the norm alone
  const long long* values;
  const unsigned char* f32;  // per tensor: float32, else bf16
  int count;
  float max_norm;
  float* norm;
  void* ws;
};
constexpr long long kMaxGradValues = 1LL << 40;  // of all tensors: their chunks are counted in 32 bits
size_t grad_norm_workspace_bytes(int count);
cudaError_t launch_grad_norm(const GradProblem& p, cudaStream_t stream);

#ifdef __CUDACC__
// A launch that `follows` may start from here on.
__device__ __forceinline__ void let_next_launch_start() { asm volatile("griddepcontrol.launch_dependents;"); }
// The exponent (of 2, biased by 127) of the least power of two s with amax / s <= 448 = 1.75 * 2^8, 2^-126
// at the least; 255, e8m0's NaN, where amax is infinite or NaN.  From amax's bits: s is
// 2^(floor(log2 amax) - 8), or twice that where the leading digits are above 1.75.
__device__ __forceinline__ uint32_t scale_exponent(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;
  const int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u);
  return (uint32_t)(e < 1 ? 1 : e);
}
// 1 / s of such an exponent: exact, as 2^(127 - e), for every e up to 253 (larger ones do not occur).
// NaN for 255, which makes every value of the block NaN.
__device__ __forceinline__ float inverse_scale(uint32_t e) {
  return e == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float((254u - e) << 23);
}
// Two values, the first in the low byte, rounded to the nearest e4m3, ties to even.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}
#endif

}  // namespace m2rnn
