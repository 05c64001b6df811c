// m2rnn_quantise.cu — bf16 or float32 values to e4m3 with a power of two for each block: activations in
// blocks of 128 along a row, weights in blocks of 128 x 128.  Memory-bound: 16 neighbouring threads take
// 128 values of a row, eight consecutive ones each, or, where rows do not start on 16-byte boundaries, a warp
// does, its lanes on neighbouring values.
// Measured, 16384 x 4096 bf16: 32 us (6.3 TB/s), 16384 x 4097: 60 us, bound by instructions there (a value a load
// and a store); weights 8192 x 4096: float32 29 us (5.8 TB/s), bf16 46, where 90 registers leave room for 16 warps an
// SM and they wait for memory.
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
// The largest |value| of 16 threads' values as bits, which order them and put NaN above all.  bf16 values keep
// to their upper halves, two to a word.
template <typename T>
__device__ __forceinline__ uint32_t top_of_16(const float (&v)[8]) {
  uint32_t top = 0;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
    return top;
  } else {
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      top = __vmaxu2(top, __byte_perm(__float_as_uint(v[i]), __float_as_uint(v[i + 1]), 0x7632) & 0x7fff7fffu);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(~0u, top, o));
    return max(top << 16, top & 0xffff0000u);
  }
}
// The largest |value| of a thread.
__device__ __forceinline__ uint32_t top_bits(const float (&v)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  return top;
}
__device__ __forceinline__ void store8(uint8_t* to, int n, const float (&v)[8], uint32_t e) {
  const float2 by = make_float2(inverse_scale(e), inverse_scale(e));
  uint32_t u[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = mul2(make_float2(v[4 * i], v[4 * i + 1]), by), b = mul2(make_float2(v[4 * i + 2], v[4 * i + 3]), by);
    u[i] = pack_e4m3x2(a.x, a.y) | pack_e4m3x2(b.x, b.y) << 16;
  }
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
                         uint8_t* __restrict__ scales, Index units, int blocks, int D) {
  let_next_launch_start();
  const Index unit = (Index)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);
  const Index row = unit / (Index)blocks;
  const int b = (int)(unit - row * (Index)blocks), at = b * kScaleBlock + (threadIdx.x & 15) * 8;
  const int n = unit < units ? max(0, min(8, D - at)) : 0;
  float v[8];
  load8(x + (n ? (long long)row * x_row + at : 0), n, true, v);
  const uint32_t e = scale_exponent(top_of_16<T>(v));
  if (n == 0) return;
  if ((threadIdx.x & 15) == 0) scales[unit] = (uint8_t)e;
  store8(q + (long long)row * q_row + at, n, v, e);
}
// Rows of whole blocks without gaps: unit u is the 128 values from 128 u on and there is no row to find.  A
// thread takes EACH units, all loaded before the first is turned.
template <typename T, int EACH>
__global__ void __launch_bounds__(kThreads) quantise_flat_kernel(const T* __restrict__ x, uint8_t* __restrict__ q,
                                                                 uint8_t* __restrict__ scales, long long units) {
  let_next_launch_start();
  const long long first = (long long)blockIdx.x * (EACH * kThreads / 16) + (threadIdx.x >> 4);
  const int piece = (threadIdx.x & 15) * 8;
  float v[EACH][8];
#pragma unroll
  for (int u = 0; u < EACH; ++u) {
    const long long unit = first + u * (kThreads / 16);
    load8(x + (unit < units ? unit * kScaleBlock + piece : 0), unit < units ? 8 : 0, true, v[u]);
  }
#pragma unroll
  for (int u = 0; u < EACH; ++u) {
    const long long unit = first + u * (kThreads / 16);
    const uint32_t e = scale_exponent(top_of_16<T>(v[u]));
    if (unit >= units) continue;
    if (piece == 0) scales[unit] = (uint8_t)e;
    store8(q + unit * kScaleBlock + piece, 8, v[u], e);
  }
}
// Two units a warp, one after the other, so that as many blocks as above take them all.
template <typename T, typename Index>
__global__ void __launch_bounds__(kThreads)
    quantise_rows_any_kernel(const T* __restrict__ x, long long x_row, uint8_t* __restrict__ q, long long q_row,
                             uint8_t* __restrict__ scales, Index units, int blocks, int D) {
  let_next_launch_start();
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const Index unit = (Index)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 5) * 2 + u;
    if (unit >= units) return;
    const Index row = unit / (Index)blocks;
    const int at = (int)(unit - row * (Index)blocks) * kScaleBlock + lane;
    const T* from = x + (long long)row * x_row;
    float v[4];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = at + 32 * i;
      if constexpr (sizeof(T) == 4)
        v[i] = c < D ? from[c] : 0.f;
      else
        v[i] = c < D ? bf16_bits_to_float(from[c]) : 0.f;
      top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    }
    const uint32_t e = scale_exponent(__reduce_max_sync(~0u, top));
    const float by = inverse_scale(e);
    if (lane == 0) scales[unit] = (uint8_t)e;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + 32 * i < D) q[(long long)row * q_row + at + 32 * i] = (uint8_t)pack_e4m3x2(v[i] * by, 0.f);
  }
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
  if (vec && D % kScaleBlock == 0 && (rows == 1 || (x_row == D && q_row == D))) {
    constexpr int kEach = sizeof(T) == 2 ? 2 : 1;  // 32 bytes of x on their way a thread
    quantise_flat_kernel<T, kEach><<<(unsigned)((grid + kEach - 1) / kEach), kThreads, 0, stream>>>(x, q, scales, units);
    return cudaGetLastError();
  }
  auto go = [&](auto index) {  // 32-bit divisions where they do: a 64-bit one costs as much as the rest
    using Index = decltype(index);
    auto* kernel = vec ? quantise_rows_kernel<T, Index> : quantise_rows_any_kernel<T, Index>;
    kernel<<<(unsigned)grid, kThreads, 0, stream>>>(x, x_row, q, q_row, scales, (Index)units, blocks, D);
    return cudaGetLastError();
  };
  return units + kThreads / 16 < 0xffffffffLL ? go(uint32_t{}) : go(0ull);
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
