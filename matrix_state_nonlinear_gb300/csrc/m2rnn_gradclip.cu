// m2rnn_gradclip.cu — the norm of all of a step's gradients together, and their scaling to at most a given
// norm.
//
//   norm = sqrt(sum over all values of g^2),   out = g min(1, max_norm / norm)
//
// Memory-bound: the norm reads every value once, the scaling reads and writes it once.  The tensors are a
// table in the launch's parameters (no copy to the device), cut into chunks that the blocks take in turn.  A
// chunk's squares are summed in float32 per thread (16 or 32 of them), everything above in 64 bits, so the
// result hardly depends on the number of values; sums that float32 cannot hold, because the values are very
// large or very small, are taken again in 64 bits.  Every block's sum has a place of its own and all are
// added in the same order by every block of the second launch: no atomics, the same bits every time.
#include <math.h>

#include "m2rnn_layer.h"
#include "ptx_util.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 512;
constexpr int kVecs = 4;                             // 16-byte accesses of a thread per chunk
constexpr int kChunkBytes = kThreads * kVecs * 16;   // 32 KB of a tensor

// One launch's tensors: entry i owns the chunks from first[i] to first[i + 1].
template <int N>
struct Table {
  int count, chunks;
  int first[N];
  unsigned long long in[N], out[N], values[N];  // values: the number of them times two, plus one for float32
};

struct Part {
  const unsigned char* in;
  unsigned char* out;
  bool f32;
  long long values;  // of this part
};

// Chunk c of the table.
template <int N>
__device__ __forceinline__ Part part_of(const Table<N>& t, int c) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  const bool f32 = t.values[lo] & 1;
  const long long each = kChunkBytes / (f32 ? 4 : 2), at = (long long)(c - t.first[lo]) * each;
  return Part{reinterpret_cast<const unsigned char*>(t.in[lo]) + at * (f32 ? 4 : 2),
              reinterpret_cast<unsigned char*>(t.out[lo]) + at * (f32 ? 4 : 2), f32,
              min(each, (long long)(t.values[lo] >> 1) - at)};
}

__device__ __forceinline__ float value(const Part& p, long long i) {
  return p.f32 ? reinterpret_cast<const float*>(p.in)[i] : bf16_bits_to_float(reinterpret_cast<const uint16_t*>(p.in)[i]);
}
__device__ __forceinline__ void put(const Part& p, long long i, float v) {
  if (p.f32)
    reinterpret_cast<float*>(p.out)[i] = v;
  else
    reinterpret_cast<uint16_t*>(p.out)[i] = f_to_bf16(v);
}
// Values before the first 16-byte boundary.
__device__ __forceinline__ int head_of(const Part& p) {
  const int size = p.f32 ? 4 : 2;
  return (int)min(p.values, (long long)((16u - ((uint32_t)(uintptr_t)p.in & 15u)) & 15u) / size);
}

__device__ __forceinline__ float squares(const uint4& u, bool f32) {
  float2 s;
  if (f32) {
    const float2 a = make_float2(__uint_as_float(u.x), __uint_as_float(u.y)), b = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
    s = fma2(a, a, mul2(b, b));
  } else {
    const float2 a = bf16x2_to_float2(u.x), b = bf16x2_to_float2(u.y), c = bf16x2_to_float2(u.z), d = bf16x2_to_float2(u.w);
    s = fma2(a, a, mul2(b, b));
    s = add2(s, fma2(c, c, mul2(d, d)));
  }
  return s.x + s.y;
}
__device__ __noinline__ double squares64(uint4 u, bool f32) {
  double s = 0;
  const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const double a = f32 ? __uint_as_float(v[i]) : bf16_lo(v[i]), b = f32 ? 0.f : bf16_hi(v[i]);
    s += a * a + b * b;
  }
  return s;
}
// Whether a sum of at most 32 squares lost something to float32's range: above it, or so small that squares
// below 2^-126 count.
__device__ __forceinline__ bool out_of_range(float s) { return !(s < INFINITY) || s < 0x1p-100f; }

// Sum over the block, for every thread, in a fixed order.  Only one warp adds in 64 bits: an SM adds two
// doubles a cycle, and 512 threads' shuffles and sums took 11 us of its time.
__device__ __forceinline__ double block_sum(double s) {
  __shared__ double part[kThreads];
  __shared__ double total;
  part[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    s = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += part[threadIdx.x + 32 * w];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    if (threadIdx.x == 0) total = s;
  }
  __syncthreads();
  return total;
}

template <int N>
__global__ void __launch_bounds__(kThreads) sum_squares_kernel(const __grid_constant__ Table<N> t, double* sums) {
  double sum = 0;
  for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const Part p = part_of(t, c);
    const int head = head_of(p), size = p.f32 ? 4 : 2, per = 16 / size;
    const long long vecs = (p.values - head) / per;
    const uint4* v = reinterpret_cast<const uint4*>(p.in + head * size);
    uint4 u[kVecs];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int at = threadIdx.x + i * kThreads;
      u[i] = at < vecs ? v[at] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) s += squares(u[i], p.f32);
    if (out_of_range(s)) {
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < kVecs; ++i) any |= u[i].x | u[i].y | u[i].z | u[i].w;
      if (any & 0x7fff7fffu)
#pragma unroll
        for (int i = 0; i < kVecs; ++i) sum += squares64(u[i], p.f32);
    } else {
      sum += s;
    }
    // The values around the 16-byte accesses: at most 7 before and 7 behind.
    const long long edge = p.values - vecs * per;
    if (threadIdx.x < edge) {
      const double x = value(p, threadIdx.x < head ? threadIdx.x : vecs * per + threadIdx.x);
      sum += x * x;
    }
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) sums[blockIdx.x] = sum;
}

// The norm from all blocks' sums, for every thread of the block.
__device__ __forceinline__ double norm_of(const double* sums, int count) {
  __shared__ double norm;
  if (threadIdx.x < 32) {
    double s = 0;
    for (int i = threadIdx.x; i < count; i += 32) s += sums[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    if (threadIdx.x == 0) norm = sqrt(s);
  }
  __syncthreads();
  return norm;
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double* sums, int count, float* norm) {
  const double n = norm_of(sums, count);
  if (threadIdx.x == 0) *norm = (float)n;
}

// Chunks from the last to the first: the last ones read are still in L2.
template <int N>
__global__ void __launch_bounds__(kThreads)
    clip_kernel(const __grid_constant__ Table<N> t, const double* sums, int count, float max_norm, float* norm,
                bool in_place) {
  const double n = norm_of(sums, count);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
  // A norm that is infinite or NaN clips nothing.
  const bool clips = n > max_norm && n < INFINITY;
  if (in_place && !clips) return;
  const float by = clips ? (float)(max_norm / n) : 1.f;
  for (int c = t.chunks - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
    const Part p = part_of(t, c);
    const int size = p.f32 ? 4 : 2, per = 16 / size;
    const bool same = (((uint32_t)(uintptr_t)p.in ^ (uint32_t)(uintptr_t)p.out) & 15u) == 0;
    const int head = same ? head_of(p) : 0;
    const long long vecs = same ? (p.values - head) / per : 0;
    const uint4* v = reinterpret_cast<const uint4*>(p.in + head * size);
    uint4* o = reinterpret_cast<uint4*>(p.out + head * size);
    uint4 u[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int at = threadIdx.x + i * kThreads;
      if (at < vecs) u[i] = v[at];
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int at = threadIdx.x + i * kThreads;
      if (at >= vecs) break;
      const float2 b = make_float2(by, by);
      uint32_t* w = &u[i].x;
      if (p.f32) {
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const float2 x = mul2(make_float2(__uint_as_float(w[j]), __uint_as_float(w[j + 1])), b);
          w[j] = __float_as_uint(x.x), w[j + 1] = __float_as_uint(x.y);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = mul2(bf16x2_to_float2(w[j]), b);
          w[j] = pack_bf16x2(x.x, x.y);
        }
      }
      o[at] = u[i];
    }
    for (long long i = threadIdx.x; i < p.values - vecs * per; i += kThreads) {
      const long long at = i < head ? i : vecs * per + i;
      put(p, at, value(p, at) * by);
    }
  }
}

constexpr int kSmall = 96, kLarge = 1000;  // tensors per launch: parameters of 2.7 and 28 KB
constexpr int kBlocks = 152 * 4;

int launches(int count) { return (count + kLarge - 1) / kLarge; }

template <int N>
void fill(Table<N>& t, const GradProblem& p, int from, int count) {
  t.count = 0, t.chunks = 0;
  for (int i = from; i < from + count; ++i) {
    if (p.values[i] == 0) continue;
    const long long each = kChunkBytes / (p.f32[i] ? 4 : 2);
    t.first[t.count] = t.chunks;
    t.in[t.count] = reinterpret_cast<uintptr_t>(p.in[i]);
    t.out[t.count] = reinterpret_cast<uintptr_t>(p.out ? p.out[i] : nullptr);
    t.values[t.count] = (unsigned long long)p.values[i] * 2 + (p.f32[i] ? 1 : 0);
    t.chunks += (int)((p.values[i] + each - 1) / each);
    ++t.count;
  }
}

// Adds its blocks' number to `parts`.
template <int N>
cudaError_t sum_squares(const GradProblem& p, int from, int count, double* sums, int* parts, cudaStream_t stream) {
  Table<N> t;
  fill(t, p, from, count);
  if (t.chunks == 0) return cudaSuccess;
  const int blocks = t.chunks < kBlocks ? t.chunks : kBlocks;
  sum_squares_kernel<N><<<blocks, kThreads, 0, stream>>>(t, sums + *parts);
  *parts += blocks;
  return cudaGetLastError();
}
template <int N>
cudaError_t clip(const GradProblem& p, int from, int count, const double* sums, int parts, bool in_place,
                 cudaStream_t stream) {
  Table<N> t;
  fill(t, p, from, count);
  const int blocks = t.chunks < kBlocks ? (t.chunks > 0 ? t.chunks : 1) : kBlocks;
  clip_kernel<N><<<blocks, kThreads, 0, stream>>>(t, sums, parts, p.max_norm, from == 0 ? p.norm : nullptr, in_place);
  return cudaGetLastError();
}

}  // namespace

size_t grad_norm_workspace_bytes(int count) { return sizeof(double) * kBlocks * (size_t)(count > 0 ? launches(count) : 0); }

cudaError_t launch_grad_norm(const GradProblem& p, cudaStream_t stream) {
  if (p.count == 0) return cudaMemsetAsync(p.norm, 0, sizeof(float), stream);
  double* sums = static_cast<double*>(p.ws);
  int parts = 0;
  cudaError_t err = cudaSuccess;
  for (int from = 0; from < p.count && err == cudaSuccess; from += kLarge) {
    const int n = p.count - from < kLarge ? p.count - from : kLarge;
    err = n <= kSmall ? sum_squares<kSmall>(p, from, n, sums, &parts, stream)
                      : sum_squares<kLarge>(p, from, n, sums, &parts, stream);
  }
  if (err != cudaSuccess) return err;
  if (!p.out) {
    norm_kernel<<<1, kThreads, 0, stream>>>(sums, parts, p.norm);
    return cudaGetLastError();
  }
  bool in_place = true;
  for (int i = 0; i < p.count; ++i) in_place = in_place && p.in[i] == p.out[i];
  for (int from = 0; from < p.count && err == cudaSuccess; from += kLarge) {
    const int n = p.count - from < kLarge ? p.count - from : kLarge;
    err = n <= kSmall ? clip<kSmall>(p, from, n, sums, parts, in_place, stream)
                      : clip<kLarge>(p, from, n, sums, parts, in_place, stream);
  }
  return err;
}

}  // namespace m2rnn
