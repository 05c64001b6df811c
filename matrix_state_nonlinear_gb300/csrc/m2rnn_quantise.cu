// m2rnn_quantise.cu — bf16 or float32 values to e4m3 with a power of two for each block: activations in
// blocks of 128 along a row, weights in blocks of 128 x 128.  Memory-bound: 16 neighbouring threads take
// 128 values of a row, eight each.
#include "m2rnn_layer.h"
#include "ptx_util.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 256;

// Eight values of which `n` exist (the others zero); aligned ones of all eight 16 bytes at a time.
__device__ __forceinline__ void load8(const float* p, int n, bool vec, float (&v)[8]) {
  if (vec && n == 8) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.f;
  }
}
__device__ __forceinline__ void load8(const uint16_t* p, int n, bool vec, float (&v)[8]) {
  if (vec && n == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? bf16_bits_to_float(p[i]) : 0.f;
  }
}
// The largest |value| as bits, which order them and put NaN above all.
__device__ __forceinline__ uint32_t top_bits(const float (&v)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  return top;
}
__device__ __forceinline__ void store8(uint8_t* to, int n, const float (&v)[8], uint32_t e) {
  const float by = inverse_scale(e);
  uint32_t u[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    u[i] = pack_e4m3x2(v[4 * i] * by, v[4 * i + 1] * by) | pack_e4m3x2(v[4 * i + 2] * by, v[4 * i + 3] * by) << 16;
  if (n == 8) {
    *reinterpret_cast<uint2*>(to) = make_uint2(u[0], u[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) to[i] = (uint8_t)(u[i >> 2] >> (8 * (i & 3)));
  }
}

// Units are (row, block of 128), counted in Index.
template <typename T, typename Index>
__global__ void __launch_bounds__(kThreads)
    quantise_rows_kernel(const T* __restrict__ x, long long x_row, uint8_t* __restrict__ q, long long q_row,
                         uint8_t* __restrict__ scales, Index units, int blocks, int D, bool vec) {
  const Index unit = (Index)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);
  const Index row = unit / (Index)blocks;
  const int b = (int)(unit - row * (Index)blocks), at = b * kScaleBlock + (threadIdx.x & 15) * 8;
  const int n = unit < units ? max(0, min(8, D - at)) : 0;
  float v[8];
  load8(x + (n ? (long long)row * x_row + at : 0), n, vec, v);
  uint32_t top = top_bits(v);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
  if (n == 0) return;
  const uint32_t e = scale_exponent(top);
  if ((threadIdx.x & 15) == 0) scales[unit] = (uint8_t)e;
  store8(q + (long long)row * q_row + at, n, v, e);
}

// One block of threads takes one block of the weights: rows 16 apart in a thread's registers.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    quantise_weight_kernel(const T* __restrict__ w, long long w_row, uint8_t* __restrict__ q, long long q_row,
                           uint8_t* __restrict__ scales, int N, int K, bool vec) {
  __shared__ uint32_t part[kThreads / 32];
  const int kb = scale_blocks(K), at = (int)(blockIdx.x % kb) * kScaleBlock + (threadIdx.x & 15) * 8;
  const long long row0 = (long long)(blockIdx.x / kb) * kScaleBlock + (threadIdx.x >> 4);
  constexpr int kEach = kScaleBlock / (kThreads / 16);
  float v[kEach][8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const long long row = row0 + i * (kThreads / 16);
    const int n = row < N ? max(0, min(8, K - at)) : 0;
    load8(w + (n ? row * w_row + at : 0), n, vec, v[i]);
    top = max(top, top_bits(v[i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) top = max(top, part[i]);
  const uint32_t e = scale_exponent(top);
  if (threadIdx.x == 0) scales[blockIdx.x] = (uint8_t)e;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const long long row = row0 + i * (kThreads / 16);
    const int n = row < N ? max(0, min(8, K - at)) : 0;
    if (n) store8(q + row * q_row + at, n, v[i], e);
  }
}

template <typename T>
cudaError_t rows_typed(const T* x, long long x_row, uint8_t* q, long long q_row, uint8_t* scales, long long rows, int D,
                       cudaStream_t stream) {
  const int blocks = scale_blocks(D);
  const long long units = rows * blocks, grid = (units + kThreads / 16 - 1) / (kThreads / 16);
  const bool vec = aligned_to(x, 16) && x_row * (int)sizeof(T) % 16 == 0;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (units + kThreads / 16 < 0xffffffffLL)  // 32-bit divisions: a 64-bit one costs as much as the rest
    quantise_rows_kernel<T, uint32_t>
        <<<(unsigned)grid, kThreads, 0, stream>>>(x, x_row, q, q_row, scales, (uint32_t)units, blocks, D, vec);
  else
    quantise_rows_kernel<T, unsigned long long>
        <<<(unsigned)grid, kThreads, 0, stream>>>(x, x_row, q, q_row, scales, units, blocks, D, vec);
  return cudaGetLastError();
}

template <typename T>
cudaError_t weight_typed(const T* w, long long w_row, uint8_t* q, long long q_row, uint8_t* scales, int N, int K,
                         cudaStream_t stream) {
  const long long grid = (long long)scale_blocks(N) * scale_blocks(K);
  const bool vec = aligned_to(w, 16) && w_row * (int)sizeof(T) % 16 == 0;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  quantise_weight_kernel<T><<<(unsigned)grid, kThreads, 0, stream>>>(w, w_row, q, q_row, scales, N, K, vec);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantise_rows(const void* x, bool f32, long long x_row, uint8_t* q, long long q_row,
                                 uint8_t* scales, long long rows, int D, cudaStream_t stream) {
  return f32 ? rows_typed(static_cast<const float*>(x), x_row, q, q_row, scales, rows, D, stream)
             : rows_typed(static_cast<const uint16_t*>(x), x_row, q, q_row, scales, rows, D, stream);
}
cudaError_t launch_quantise_weight(const void* w, bool f32, long long w_row, uint8_t* q, long long q_row,
                                   uint8_t* scales, int N, int K, cudaStream_t stream) {
  return f32 ? weight_typed(static_cast<const float*>(w), w_row, q, q_row, scales, N, K, stream)
             : weight_typed(static_cast<const uint16_t*>(w), w_row, q, q_row, scales, N, K, stream);
}

}  // namespace m2rnn
