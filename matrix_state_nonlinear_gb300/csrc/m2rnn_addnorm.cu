// m2rnn_addnorm.cu — the residual's addition with the RMS norm in front of a block, its 8-bit form and
// its backward.
//
//   h = stream + x (rounded to the stream's type),  inv = 1 / sqrt(mean(h^2) + eps),  out = h inv w
// Backward, with g = dout w and dh the gradient that arrives at h from behind:
//   d = dh + inv g - h inv^3 mean(g h)  (dx and dresidual),  dw = sum over rows of dout h inv
//
// Memory-bound.  A block takes one row, held in registers, eight channels of a thread to a chunk, so that every
// input is read once; the norm is taken of h as the stream's type holds it, which is what the next layer and the
// backward read.  Where everything is 16-byte aligned (VEC) the eight are consecutive, and in 8 bits 16
// neighbouring threads hold the 128 channels of a scale.  Otherwise they lie a block's threads apart, so that a
// warp's accesses are still of consecutive values, and the 128 are those of four warps.
// Measured: 65536 x 2048, bf16: forward 153 us (7.0 TB/s, 1.03 of a copy's rate), backward 174 us with the sums.
#include "m2rnn_layer.h"
#include "ptx_util.cuh"

namespace m2rnn {
namespace {

__device__ __forceinline__ float2 pair(float x) { return make_float2(x, x); }

// Chunk r of a thread's channels of a row of D, as loaded, so that a load can be started ahead of its use.
// Channels that are not there are zero and are not stored.
template <typename T, bool VEC>
struct Raw8 {
  uint4 u[sizeof(T) / 2];
  // Without VEC: channel i of the chunk.
  static __device__ __forceinline__ int channel(int r, int i) { return (8 * r + i) * blockDim.x + threadIdx.x; }
  static __device__ __forceinline__ int first(int r) { return 8 * (threadIdx.x + r * blockDim.x); }
  __device__ __forceinline__ void load(const T* row, int r, int D) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i)
        u[i] = first(r) < D ? reinterpret_cast<const uint4*>(row + first(r))[i] : make_uint4(0, 0, 0, 0);
    } else {
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = channel(r, i);
        if constexpr (sizeof(T) == 4)
          v[i] = c < D ? __float_as_uint(row[c]) : 0u;
        else
          v[i] = c < D ? row[c] : 0u;
      }
      if constexpr (sizeof(T) == 4) {
        u[0] = make_uint4(v[0], v[1], v[2], v[3]);
        u[sizeof(T) / 2 - 1] = make_uint4(v[4], v[5], v[6], v[7]);
      } else {
        u[0] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
      }
    }
  }
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[2 * i] = make_float2(__uint_as_float(u[i].x), __uint_as_float(u[i].y));
        f[2 * i + 1] = make_float2(__uint_as_float(u[i].z), __uint_as_float(u[i].w));
      }
    } else {
      f[0] = bf16x2_to_float2(u[0].x), f[1] = bf16x2_to_float2(u[0].y);
      f[2] = bf16x2_to_float2(u[0].z), f[3] = bf16x2_to_float2(u[0].w);
    }
  }
  __device__ __forceinline__ void set(const float2 (&f)[4]) {  // rounded to T
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        u[i] = make_uint4(__float_as_uint(f[2 * i].x), __float_as_uint(f[2 * i].y), __float_as_uint(f[2 * i + 1].x),
                          __float_as_uint(f[2 * i + 1].y));
    } else {
      u[0] = make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                        pack_bf16x2(f[3].x, f[3].y));
    }
  }
  __device__ __forceinline__ void store(T* row, int r, int D) const {
    if constexpr (VEC) {
      if (first(r) < D)
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(row + first(r))[i] = u[i];
    } else {
      const uint4 a = u[0], b = u[sizeof(T) / 2 - 1];
      const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = channel(r, i);
        if constexpr (sizeof(T) == 4) {
          if (c < D) row[c] = __uint_as_float(v[i]);
        } else {
          if (c < D) row[c] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
        }
      }
    }
  }
};

// Sums of two values over the block, for every thread.  `turn` (0, 1, 0, ...) chooses the scratch, so that
// one barrier a sum is enough.
__device__ __forceinline__ float2 block_sum(float2 s, int turn) {
  __shared__ float2 part[2][16];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    s = add2(s, make_float2(__shfl_xor_sync(~0u, s.x, o), __shfl_xor_sync(~0u, s.y, o)));
  const int warps = blockDim.x >> 5;
  if (warps > 1) {
    if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = s;
    __syncthreads();
    s = part[turn][0];
    for (int w = 1; w < warps; ++w) s = add2(s, part[turn][w]);
  }
  return s;
}

// |values| as bits, which order them and put NaN above all.
__device__ __forceinline__ uint32_t bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Chunk r of a row in 8 bits, VEC: 16 threads to a scale.
__device__ __forceinline__ void store_fp8(const float2 (&v)[4], int r, int D, uint8_t* q, uint8_t* scales) {
  uint32_t top = 0, b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(bits(v[i].x), bits(v[i].y)));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
  const uint32_t e = scale_exponent(top);
  const float2 by = pair(inverse_scale(e));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = mul2(v[i], by);
    b[i] = pack_e4m3x2(y.x, y.y);
  }
  const int c = 8 * (threadIdx.x + r * blockDim.x);
  if (c >= D) return;
  if (c % kScaleBlock == 0) scales[c / kScaleBlock] = (uint8_t)e;
  *reinterpret_cast<uint2*>(q + c) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
}
// A row in 8 bits without VEC: a block has a multiple of 128 threads, so that the 128 channels of a scale are
// one value of each thread of four warps.
template <int R>
__device__ __forceinline__ void store_fp8_any(const float2 (&v)[R][4], int D, uint8_t* q, uint8_t* scales) {
  __shared__ uint32_t tops[8 * R][16];
  const int warp = threadIdx.x >> 5;
  const float* value = &v[0][0].x;
#pragma unroll
  for (int i = 0; i < 8 * R; ++i) {
    const uint32_t top = __reduce_max_sync(~0u, bits(value[i]));
    if ((threadIdx.x & 31) == 0) tops[i][warp] = top;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8 * R; ++i) {
    const uint32_t* t = &tops[i][warp & ~3];
    const uint32_t e = scale_exponent(max(max(t[0], t[1]), max(t[2], t[3])));
    const int c = i * blockDim.x + threadIdx.x;
    if (c < D) {
      if (c % kScaleBlock == 0) scales[c / kScaleBlock] = (uint8_t)e;
      q[c] = (uint8_t)pack_e4m3x2(value[i] * inverse_scale(e), 0.f);
    }
  }
}

template <typename T, bool FP8, bool VEC, int R>
__global__ void __launch_bounds__(512)
    add_rmsnorm_kernel(AddNormProblem p, uint16_t* __restrict__ out, uint8_t* __restrict__ q, long long q_row,
                       uint8_t* __restrict__ scales) {
  const float inv_d = 1.f / (float)p.D;
  int turn = 0;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    const T* stream = static_cast<const T*>(p.stream) + row * p.stream_row;
    const uint16_t* x = p.x ? p.x + row * p.x_row : nullptr;
    float2 h[R][4], s = pair(0.f);
    Raw8<T, VEC> a[R];
    Raw8<uint16_t, VEC> b[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      a[r].load(stream, r, p.D);
      if (x) b[r].load(x, r, p.D);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      a[r].get(h[r]);
      if (x) {
        float2 v[4];
        b[r].get(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[r][i] = add2(h[r][i], v[i]);
        a[r].set(h[r]);
        if (sizeof(T) == 2) a[r].get(h[r]);
      }
      if (p.h) a[r].store(static_cast<T*>(p.h) + row * p.D, r, p.D);
#pragma unroll
      for (int i = 0; i < 4; ++i) s = fma2(h[r][i], h[r][i], s);
    }
    const float inv = rsqrtf(block_sum(make_float2(s.x + s.y, 0.f), turn).x * inv_d + p.eps);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      Raw8<float, VEC> u;
      float2 w[4];
      u.load(p.w, r, p.D);
      u.get(w);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[r][i] = mul2(mul2(h[r][i], pair(inv)), w[i]);
      if constexpr (FP8 && VEC) {
        store_fp8(h[r], r, p.D, q + row * q_row, scales + row * scale_blocks(p.D));
      } else if constexpr (!FP8) {
        Raw8<uint16_t, VEC> o;
        o.set(h[r]);
        o.store(out + row * p.D, r, p.D);
      }
    }
    if constexpr (FP8 && !VEC) store_fp8_any<R>(h, p.D, q + row * q_row, scales + row * scale_blocks(p.D));
  }
}

// 16 bytes to shared memory without passing through registers, by way of L1 (SECTORS: where a thread's next
// copy is the other half of the sector); a thread's own copies are complete once at most N of its later groups
// are not.
template <bool SECTORS>
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  if constexpr (SECTORS)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The rows of h, dout and dh that a block reads, on their way ahead of their use: kAhead rows in shared memory,
// where each thread reads what it has copied itself (no barrier), or, at any alignment, one row in registers.
// Four rows for a bf16 stream of up to 8192 channels; as many of a float32 one would leave room for half the
// blocks on an SM (65536 x 2048: 417 us instead of 325 with two).
template <typename T, int R>
constexpr int kAhead = R * sizeof(T) <= 4 && sizeof(T) == 2 ? 4 : R * sizeof(T) <= 8 ? 2 : 1;
template <typename T, int R>
constexpr int kRingPerThread = kAhead<T, R> * (2 * (int)sizeof(T) / 2 + 1) * R * 16;  // bytes
template <typename T, bool VEC, int R>
struct RowStream {
  static constexpr int kRows = kAhead<T, R>, kParts = sizeof(T) / 2;  // 16-byte pieces of 8 values
  const AddNormBackwardProblem& p;
  uint4* own;  // [kRows][kParts + 1 + kParts][R][threads]
  int at = 0, to = 0;
  Raw8<T, VEC> hr[R], er[R];
  Raw8<uint16_t, VEC> dr[R];

  __device__ __forceinline__ RowStream(const AddNormBackwardProblem& p_, uint4* smem) : p(p_), own(smem + threadIdx.x) {}
  __device__ __forceinline__ uint4* slot(int stage, int part, int r) const {
    return own + ((stage * (2 * kParts + 1) + part) * R + r) * blockDim.x;
  }
  __device__ __forceinline__ void start(long long row) {
    if (row < p.rows) {
      const T *h = static_cast<const T*>(p.h) + row * p.D, *e = static_cast<const T*>(p.dh) + row * p.D;
      const uint16_t* d = p.dout + row * p.D;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if constexpr (VEC) {
          const int c = Raw8<T, VEC>::first(r);
          if (c < p.D) {
#pragma unroll
            for (int k = 0; k < kParts; ++k)
              copy16<kParts == 2>(smem_u32(slot(to, k, r)), reinterpret_cast<const uint4*>(h + c) + k);
            copy16<false>(smem_u32(slot(to, kParts, r)), d + c);
            if (p.dh)
#pragma unroll
              for (int k = 0; k < kParts; ++k)
                copy16<kParts == 2>(smem_u32(slot(to, kParts + 1 + k, r)), reinterpret_cast<const uint4*>(e + c) + k);
          }
        } else {
          hr[r].load(h, r, p.D);
          dr[r].load(d, r, p.D);
          if (p.dh) er[r].load(e, r, p.D);
        }
      }
    }
    if constexpr (VEC) {
      copies_commit();
      to = to + 1 == kRows ? 0 : to + 1;
    }
  }
  __device__ __forceinline__ void begin(long long row, long long step) {
#pragma unroll
    for (int i = 0; i < (VEC ? kRows - 1 : kParts / kParts); ++i) start(row + i * step);
  }
  // dh of the row at hand is taken before the sums where there is room to hold it across them (65536 x 2048
  // float32: 317 us, 364 where it is taken after them; 4000 x 16384 bf16: 215 and 124).
  static constexpr bool kEarly = VEC && R <= 2;
  // h, dout and, if early, dh of `row`, zeros behind the last channel; a later row starts.
  __device__ __forceinline__ void next(long long row, long long step, float2 (&h)[R][4], float2 (&d)[R][4],
                                       float2 (&e)[R][4]) {
    if constexpr (VEC) {
      start(row + (kRows - 1) * step);
      copies_wait<kRows - 1>();
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int i = 0; i < 4; ++i) h[r][i] = d[r][i] = e[r][i] = pair(0.f);
      if (!VEC || Raw8<T, VEC>::first(r) < p.D) {
        if constexpr (VEC) {
#pragma unroll
          for (int k = 0; k < kParts; ++k) hr[r].u[k] = *slot(at, k, r);
          dr[r].u[0] = *slot(at, kParts, r);
          if (kEarly && p.dh)
#pragma unroll
            for (int k = 0; k < kParts; ++k) er[r].u[k] = *slot(at, kParts + 1 + k, r);
        }
        hr[r].get(h[r]);
        dr[r].get(d[r]);
        if (kEarly && p.dh) er[r].get(e[r]);
      }
    }
  }
  // dh of chunk r, where it is late.
  __device__ __forceinline__ void late(int r, float2 (&e)[4]) {
    if (kEarly || !p.dh || (VEC && Raw8<T, VEC>::first(r) >= p.D)) return;
    if constexpr (VEC)
#pragma unroll
      for (int k = 0; k < kParts; ++k) er[r].u[k] = *slot(at, kParts + 1 + k, r);
    er[r].get(e);
  }
  __device__ __forceinline__ void done(long long row, long long step) {
    if constexpr (VEC)
      at = at + 1 == kRows ? 0 : at + 1;
    else
      start(row + step);
  }
};

// Block b takes rows b, + blocks, ...; its channels' part of dw adds up in registers and goes to row b of
// `part`.
template <typename T, bool VEC, int R>
__global__ void __launch_bounds__(512, R == 1 ? 2 : 1)
    add_rmsnorm_backward_kernel(AddNormBackwardProblem p, float* __restrict__ part) {
  extern __shared__ uint4 ring[];
  const float inv_d = 1.f / (float)p.D;
  constexpr bool kKeep = R <= 2;  // the weight stays in registers where there is room for it
  float2 dw[R][4], kept[kKeep ? R : 1][4];
  auto weight = [&](int r, float2(&w)[4]) {
    Raw8<float, VEC> u;
    u.load(p.w, r, p.D);
    u.get(w);
  };
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if constexpr (kKeep) weight(r, kept[r]);
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[r][i] = pair(0.f);
  }
  RowStream<T, VEC, R> rows(p, ring);
  rows.begin(blockIdx.x, gridDim.x);
  int turn = 0;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    float2 h[R][4], d[R][4], s1 = pair(0.f), s2 = pair(0.f);
    float2 e[R][4];
    rows.next(row, gridDim.x, h, d, e);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 w[4];
      if constexpr (!kKeep) weight(r, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s1 = fma2(h[r][i], h[r][i], s1);
        s2 = fma2(mul2(d[r][i], kKeep ? kept[kKeep ? r : 0][i] : w[i]), h[r][i], s2);
      }
    }
    const float2 sum = block_sum(make_float2(s1.x + s1.y, s2.x + s2.y), turn);
    const float inv = rsqrtf(sum.x * inv_d + p.eps);
    const float2 iv = pair(inv), back = pair(-inv * inv * inv * (sum.y * inv_d));
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 o[4], w[4];
      rows.late(r, e[r]);
      if constexpr (!kKeep) weight(r, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dw[r][i] = fma2(d[r][i], mul2(h[r][i], iv), dw[r][i]);
        o[i] = add2(fma2(h[r][i], back, mul2(mul2(d[r][i], kKeep ? kept[kKeep ? r : 0][i] : w[i]), iv)), e[r][i]);
      }
      if (p.dx) {
        Raw8<uint16_t, VEC> u;
        u.set(o);
        u.store(p.dx + row * p.D, r, p.D);
      }
      if (p.dresidual) {
        Raw8<T, VEC> u;
        u.set(o);
        u.store(static_cast<T*>(p.dresidual) + row * p.D, r, p.D);
      }
    }
    rows.done(row, gridDim.x);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    Raw8<float, VEC> u;
    u.set(dw[r]);
    u.store(part + (long long)blockIdx.x * p.D, r, p.D);
  }
}

// Threads of a row's block for R chunks per thread: whole warps, without VEC four at a time.
int threads_for(int D, int R, bool vec) {
  const int chunks = (D + 7) / 8, whole = vec ? 32 : 128;
  return ((chunks + R - 1) / R + whole - 1) / whole * whole;
}
// Chunks per thread, the fewest from `least` on whose block has at most 512 threads.
int chunks_each(int D, int least) {
  int R = least;
  while (threads_for(D, R, true) > 512) R *= 2;
  return R;
}

template <int N>
struct Int {
  static constexpr int value = N;
};
template <typename F>
cudaError_t with_chunks(int R, F f) {
  return R == 1 ? f(Int<1>{}) : R == 2 ? f(Int<2>{}) : f(Int<4>{});
}

template <typename T, bool FP8, bool VEC>
cudaError_t forward(const AddNormProblem& p, uint16_t* out, uint8_t* q, long long q_row, uint8_t* scales,
                    cudaStream_t stream) {
  // Few rows are spread as wide as they go; of many, two chunks a thread (65536 x 2048: 153 us; one chunk
  // 169, four 158; 8191 x 4096 in 8 bits: 58, 65, 64).
  const int R = chunks_each(p.D, VEC && p.rows >= 152 * 16 ? 2 : 1);
  return with_chunks(R, [&](auto r) {
    constexpr int N = decltype(r)::value;
    const unsigned blocks = (unsigned)(p.rows < 0x7fffffff ? p.rows : 0x7fffffff);
    add_rmsnorm_kernel<T, FP8, VEC, N><<<blocks, threads_for(p.D, N, VEC), 0, stream>>>(p, out, q, q_row, scales);
    return cudaGetLastError();
  });
}

bool rows_of_8(const void* p, long long row, size_t size) { return aligned_to(p, 16) && row * size % 16 == 0; }

bool vec_ok(const AddNormProblem& p) {
  const size_t size = p.stream_f32 ? 4 : 2;
  return p.D % 8 == 0 && aligned_to(p.w, 16) && rows_of_8(p.stream, p.stream_row, size) &&
         (!p.x || rows_of_8(p.x, p.x_row, 2)) && aligned_to(p.h, 16);
}

template <bool FP8>
cudaError_t dispatch(const AddNormProblem& p, bool vec, uint16_t* out, uint8_t* q, long long q_row, uint8_t* scales,
                     cudaStream_t stream) {
  if (p.stream_f32)
    return vec ? forward<float, FP8, true>(p, out, q, q_row, scales, stream)
               : forward<float, FP8, false>(p, out, q, q_row, scales, stream);
  return vec ? forward<uint16_t, FP8, true>(p, out, q, q_row, scales, stream)
             : forward<uint16_t, FP8, false>(p, out, q, q_row, scales, stream);
}

// Blocks of the backward, and rows of its sums: 1024 threads for every SM.
int backward_blocks(long long rows, int D) {
  const long long most = 152LL * (1024 / threads_for(D, chunks_each(D, 1), true));
  return (int)(rows < most ? (rows > 0 ? rows : 1) : most);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const AddNormProblem& p, uint16_t* out, cudaStream_t stream) {
  return dispatch<false>(p, vec_ok(p) && aligned_to(out, 16), out, nullptr, 0, nullptr, stream);
}
cudaError_t launch_add_rmsnorm_fp8(const AddNormProblem& p, uint8_t* q, long long q_row, uint8_t* scales,
                                   cudaStream_t stream) {
  return dispatch<true>(p, vec_ok(p), nullptr, q, q_row, scales, stream);
}

size_t add_rmsnorm_backward_workspace_floats(long long rows, int D) { return (size_t)backward_blocks(rows, D) * D; }

cudaError_t launch_add_rmsnorm_backward(const AddNormBackwardProblem& p, cudaStream_t stream) {
  if (p.rows == 0) return cudaMemsetAsync(p.dw, 0, sizeof(float) * p.D, stream);
  const bool vec = p.D % 8 == 0 && aligned_to(p.w, 16) && aligned_to(p.h, 16) && aligned_to(p.dout, 16) &&
                   aligned_to(p.dh, 16) && aligned_to(p.dx, 16) && aligned_to(p.dresidual, 16);
  const int blocks = backward_blocks(p.rows, p.D);
  const cudaError_t err = with_chunks(chunks_each(p.D, 1), [&](auto r) {
    constexpr int R = decltype(r)::value;
    auto go = [&](auto kernel) {
      const int threads = threads_for(p.D, R, vec);
      const int bytes = vec ? threads * (p.stream_f32 ? kRingPerThread<float, R> : kRingPerThread<uint16_t, R>) : 0;
      // At every launch: the attribute belongs to the current device.
      const cudaError_t attr = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
      if (attr != cudaSuccess) return attr;
      kernel<<<blocks, threads, bytes, stream>>>(p, p.ws);
      return cudaGetLastError();
    };
    if (p.stream_f32)
      return vec ? go(add_rmsnorm_backward_kernel<float, true, R>) : go(add_rmsnorm_backward_kernel<float, false, R>);
    return vec ? go(add_rmsnorm_backward_kernel<uint16_t, true, R>)
               : go(add_rmsnorm_backward_kernel<uint16_t, false, R>);
  });
  if (err != cudaSuccess) return err;
  return launch_sum_rows(p.ws, p.dw, nullptr, blocks, p.D, p.D, p.D, stream);
}

}  // namespace m2rnn
