// m2rnn_gradclip.cu — the norm of all of a step's gradients together, and their scaling to at most a given
// norm.
//
//   norm = sqrt(sum over all values of g^2),   out = g min(1, max_norm / norm)
//
// Memory-bound: the norm reads every value once, the scaling reads and writes it once.  The tensors are a
// table in the launch's parameters (no copy to the device).  Those of 64 KB and more are laid end to end in units
// of 8 KB, of which every block takes an equal stretch, so that blocks end together however the tensors are cut;
// the scaling takes each stretch from its end, which the norm read last and L2 still holds.  Smaller tensors,
// each of which costs a block a whole turn whatever its size, go to the blocks one by one.
// A thread's squares are summed in float32 for one part (32 or 64 of them) and then as a pair of floats, hi and
// lo, that loses nothing; blocks' sums are 64-bit ones.  The result hardly depends on the number of values.  Sums
// that float32 cannot hold, because the values are very large or very small, are taken again in 64 bits.
// Every block's sum has a place of its own and all are added in the same order by every block of the second
// launch: no atomics, the same bits every time.
// Measured, 384M bf16 values: 361 us, the norm 128 (6.0 TB/s), the scaling 233 (6.6 TB/s).
#include <math.h>

#include "m2rnn_layer.h"
#include "ptx_util.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 512;
constexpr int kUnitBytes = kThreads * 16;
constexpr int kVecs = 8;  // units of one tensor that a block takes at once, 16 bytes a thread of each

// One launch's tensors: entry i < large owns the units from first[i] to first[i + 1], the others are small.
template <int N>
struct Table {
  int count, large, units;
  int first[N + 1];
  unsigned long long in[N], out[N], values[N];  // values: the number of them times two, plus one for float32
};

struct Part {
  const unsigned char* in;
  unsigned char* out;
  bool f32;
  long long values;  // of this part, 0 when there are no more
};

// A block's stretch of units in parts of up to kVecs units of one tensor, forwards or backwards, and then its
// small tensors.
template <int N, bool BACK>
struct Stretch {
  const Table<N>& t;
  int from, to, entry, small;
  __device__ __forceinline__ Stretch(const Table<N>& t_) : t(t_), small(t_.large + blockIdx.x) {
    from = (int)((long long)t.units * blockIdx.x / gridDim.x);
    to = (int)((long long)t.units * (blockIdx.x + 1) / gridDim.x);
    const int u = BACK ? to - 1 : from;
    int lo = 0, hi = t.large - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (t.first[mid] <= u)
        lo = mid;
      else
        hi = mid - 1;
    }
    entry = lo;
  }
  __device__ __forceinline__ Part next() {
    int i = entry, n = kVecs;
    long long off = 0;  // in units
    if (from >= to) {
      i = small, small += gridDim.x;
      if (i >= t.count) return Part{nullptr, nullptr, true, 0};
    } else if (BACK) {
      if (t.first[i] >= to) i = --entry;
      const int at = max(max(from, t.first[i]), to - kVecs);
      n = to - at, off = at - t.first[i], to = at;
    } else {
      if (t.first[i + 1] <= from) i = ++entry;
      n = min(min(to, t.first[i + 1]) - from, kVecs), off = from - t.first[i], from += n;
    }
    const bool f32 = t.values[i] & 1;
    const int size = f32 ? 4 : 2, each = kUnitBytes / size;
    return Part{reinterpret_cast<const unsigned char*>(t.in[i]) + off * kUnitBytes,
                reinterpret_cast<unsigned char*>(t.out[i]) + off * kUnitBytes, f32,
                min((long long)n * each, (long long)(t.values[i] >> 1) - off * each)};
  }
};

__device__ __forceinline__ float value(const Part& p, long long i) {
  return p.f32 ? reinterpret_cast<const float*>(p.in)[i]
               : bf16_bits_to_float(reinterpret_cast<const uint16_t*>(p.in)[i]);
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
    const float2 a = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    const float2 b = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
    s = fma2(a, a, mul2(b, b));
  } else {
    const float2 a = bf16x2_to_float2(u.x), b = bf16x2_to_float2(u.y);
    const float2 c = bf16x2_to_float2(u.z), d = bf16x2_to_float2(u.w);
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
// 16 bytes of values times `by`, in 64 bits.
__device__ __noinline__ uint4 times64(uint4 u, bool f32, double by) {
  uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = f32 ? __float_as_uint((float)(__uint_as_float(v[i]) * by))
               : pack_bf16x2((float)(bf16_lo(v[i]) * by), (float)(bf16_hi(v[i]) * by));
  return make_uint4(v[0], v[1], v[2], v[3]);
}
// Whether a sum of at most 64 squares is near the ends of float32's range: so large that a thread's sums (fewer than
// 2^20 of them for the most values that a call takes) could leave it together, or so small that squares below
// 2^-126 count.
__device__ __forceinline__ bool out_of_range(float s) { return !(s < 0x1p100f) || s < 0x1p-100f; }

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

// The 16-byte accesses of a part: their number and the first.
struct Vecs {
  int head;
  long long count;
  const uint4* in;
  uint4* out;
};
__device__ __forceinline__ Vecs vecs_of(const Part& p, bool any) {
  const int size = p.f32 ? 4 : 2, head = any ? head_of(p) : 0;
  return Vecs{head, any ? (p.values - head) * size / 16 : 0, reinterpret_cast<const uint4*>(p.in + head * size),
              reinterpret_cast<uint4*>(p.out + head * size)};
}
__device__ __forceinline__ void load(const Vecs& v, uint4 (&u)[kVecs]) {
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int at = threadIdx.x + i * kThreads;
    u[i] = at < v.count ? v.in[at] : make_uint4(0, 0, 0, 0);
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads) sum_squares_kernel(const __grid_constant__ Table<N> t, double* sums) {
  let_next_launch_start();
  Stretch<N, false> stretch(t);
  double rare = 0;
  float hi = 0.f, lo = 0.f;
  Part p = stretch.next();
  Vecs v = vecs_of(p, true);
  uint4 u[kVecs];
  load(v, u);
  while (p.values > 0) {
    const Part q = stretch.next();
    const Vecs w = vecs_of(q, true);
    uint4 ahead[kVecs];
    load(w, ahead);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) s += squares(u[i], p.f32);
    if (out_of_range(s)) {
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < kVecs; ++i) any |= u[i].x | u[i].y | u[i].z | u[i].w;
      if (any & (p.f32 ? 0x7fffffffu : 0x7fff7fffu))  // any value but zeros, whatever their signs
#pragma unroll
        for (int i = 0; i < kVecs; ++i) rare += squares64(u[i], p.f32);
    } else {  // hi + lo += s, exactly but for the rounding of lo
      const float sum = hi + s, back = sum - hi;
      lo += (hi - (sum - back)) + (s - back);
      hi = sum;
    }
    // The values around the 16-byte accesses: at most 7 before and 7 behind.
    const long long inner = v.count * (p.f32 ? 4 : 8);
    if (threadIdx.x < p.values - inner) {
      const double x = value(p, threadIdx.x < v.head ? threadIdx.x : inner + threadIdx.x);
      rare += x * x;
    }
    p = q, v = w;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) u[i] = ahead[i];
  }
  const double sum = block_sum(rare + ((double)hi + (double)lo));
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

template <int N>
__global__ void __launch_bounds__(kThreads)
    clip_kernel(const __grid_constant__ Table<N> t, const double* sums, int count, float max_norm, float* norm,
                bool in_place) {
  Stretch<N, true> stretch(t);
  // Whether 16 bytes of a part lie the same way where they are read and written.
  auto alike = [](const Part& p) { return (((uint32_t)(uintptr_t)p.in ^ (uint32_t)(uintptr_t)p.out) & 15u) == 0; };
  Part p = stretch.next();
  Vecs v = vecs_of(p, alike(p));
  uint4 u[kVecs];
  load(v, u);  // on its way while the last of the sums are made and added
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const double n = norm_of(sums, count);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
  // A norm that is infinite or NaN clips nothing.
  const bool clips = n > max_norm && n < INFINITY;
  if (in_place && !clips) return;
  const double factor = clips ? max_norm / n : 1.0;
  // Below 2^-126 float32 would hold the factor with few bits or none, and values of up to 2^128 need them.
  const bool small = factor < 0x1p-126;
  const float by = (float)factor;
  const float2 b = make_float2(by, by);
  while (p.values > 0) {
    const Part q = stretch.next();
    const Vecs w = vecs_of(q, alike(q));
    uint4 ahead[kVecs];
    load(w, ahead);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      uint32_t x[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      if (small) {
        const uint4 y = times64(u[i], p.f32, factor);
        x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
      } else if (p.f32) {
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const float2 y = mul2(make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), b);
          x[j] = __float_as_uint(y.x), x[j + 1] = __float_as_uint(y.y);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 y = mul2(bf16x2_to_float2(x[j]), b);
          x[j] = pack_bf16x2(y.x, y.y);
        }
      }
      const int at = threadIdx.x + i * kThreads;
      if (at < v.count) v.out[at] = make_uint4(x[0], x[1], x[2], x[3]);
    }
    const long long inner = v.count * (p.f32 ? 4 : 8);
    for (long long i = threadIdx.x; i < p.values - inner; i += kThreads) {
      const long long at = i < v.head ? i : inner + i;
      put(p, at, small ? (float)(value(p, at) * factor) : value(p, at) * by);
    }
    p = q, v = w;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) u[i] = ahead[i];
  }
}

constexpr int kSmall = 32, kMiddle = 320, kLarge = 1000;  // tensors per launch: parameters of 1, 9 and 28 KB
// One block an SM with 8 accesses a thread on their way (384M bf16 values: 360 us, 5.6M float32: 15.5; two
// blocks with four each 364 and 17.0, four 368 and 26.7).
constexpr int kBlocks = 152;

int launches(int count) { return (count + kLarge - 1) / kLarge; }

template <int N>
void fill(Table<N>& t, const GradProblem& p, int from, int count) {
  t.count = t.large = t.units = 0;
  for (int small = 0; small < 2; ++small) {
    for (int i = from; i < from + count; ++i) {
      const long long each = kUnitBytes / (p.f32[i] ? 4 : 2), units = (p.values[i] + each - 1) / each;
      if (units == 0 || (units <= kVecs) != (small != 0)) continue;
      t.first[t.count] = t.units;
      t.in[t.count] = reinterpret_cast<uintptr_t>(p.in[i]);
      t.out[t.count] = reinterpret_cast<uintptr_t>(p.out ? p.out[i] : nullptr);
      t.values[t.count] = (unsigned long long)p.values[i] * 2 + (p.f32[i] ? 1 : 0);
      if (!small) t.units += (int)units;
      ++t.count;
    }
    if (!small) t.large = t.count, t.first[t.count] = t.units;
  }
}
template <int N>
int blocks_of(const Table<N>& t) {
  const int most = t.units + t.count - t.large;
  return most < kBlocks ? (most > 0 ? most : 1) : kBlocks;
}

// Adds its blocks' number to `parts`.
template <int N>
cudaError_t sum_squares(const GradProblem& p, int from, int count, double* sums, int* parts, cudaStream_t stream) {
  Table<N> t;
  fill(t, p, from, count);
  if (t.count == 0) return cudaSuccess;
  const int blocks = blocks_of(t);
  sum_squares_kernel<N><<<blocks, kThreads, 0, stream>>>(t, sums + *parts);
  *parts += blocks;
  return cudaGetLastError();
}
template <int N>
cudaError_t clip(const GradProblem& p, int from, int count, const double* sums, int parts, bool in_place,
                 cudaStream_t stream) {
  Table<N> t;
  fill(t, p, from, count);
  // Starts while the launch that sums the squares ends, and waits for it before it reads sums or writes anything.
  // Behind another of its kind (more tensors than a launch takes) it starts after that.
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(blocks_of(t));
  c.blockDim = dim3(kThreads);
  c.stream = stream;
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &a;
  c.numAttrs = from == 0 ? 1 : 0;
  return cudaLaunchKernelEx(&c, clip_kernel<N>, t, sums, parts, p.max_norm, from == 0 ? p.norm : nullptr, in_place);
}

}  // namespace

size_t grad_norm_workspace_bytes(int count) {
  return sizeof(double) * kBlocks * (size_t)(count > 0 ? launches(count) : 0);
}

cudaError_t launch_grad_norm(const GradProblem& p, cudaStream_t stream) {
  if (p.count == 0) return cudaMemsetAsync(p.norm, 0, sizeof(float), stream);
  double* sums = static_cast<double*>(p.ws);
  int parts = 0;
  cudaError_t err = cudaSuccess;
  for (int from = 0; from < p.count && err == cudaSuccess; from += kLarge) {
    const int n = p.count - from < kLarge ? p.count - from : kLarge;
    err = n <= kSmall    ? sum_squares<kSmall>(p, from, n, sums, &parts, stream)
          : n <= kMiddle ? sum_squares<kMiddle>(p, from, n, sums, &parts, stream)
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
    err = n <= kSmall    ? clip<kSmall>(p, from, n, sums, parts, in_place, stream)
          : n <= kMiddle ? clip<kMiddle>(p, from, n, sums, parts, in_place, stream)
                         : clip<kLarge>(p, from, n, sums, parts, in_place, stream);
  }
  return err;
}

}  // namespace m2rnn
