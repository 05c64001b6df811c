// m2rnn_addnorm.cu — the residual's addition with the RMS norm in front of a block, its 8-bit form and
// its backward.
//
//   h = stream + x (rounded to the stream's type),  inv = 1 / sqrt(mean(h^2) + eps),  out = h inv w
// Backward, with g = dout w and dh the gradient that arrives at h from behind:
//   d = dh + inv g - h inv^3 mean(g h)  (dx and dresidual),  dw = sum over rows of dout h inv
//
// Memory-bound.  A block takes one row, held in registers, eight channels of a thread to a chunk, so that every
// input is read once; half a warp or a warp takes a row of few channels, and a block several of those.  The norm
// is taken of h as the stream's type holds it, which is what the next layer and the backward read.  Chunks are
// eight consecutive channels where memory allows 16-byte accesses (and in 8 bits 16 neighbouring threads hold the
// 128 channels of a scale); otherwise they lie a row's threads apart, so that a warp's accesses are still of
// consecutive values.
// Measured: 65536 x 2048, bf16: forward 154 us (7.0 TB/s, 1.03 of a copy's rate), backward 171 us with the sums;
// 8191 x 4096 in 8 bits on a float32 stream: 56 us (6.6 TB/s); 65536 bf16 rows of 1001: 102 and 107 us, of 1000 77
// and 105; backward of wide rows, 3000 x 9001: 108 us (bf16) and 140 (float32).
#include "m2rnn_layer.h"
#include "ptx_util.cuh"

namespace m2rnn {
namespace {

template <int N>
struct Int {
  static constexpr int value = N;
};

__device__ __forceinline__ float2 pair(float x) { return make_float2(x, x); }

// How a row lies in memory.  kVec: every row of every tensor starts on 16 bytes.  kShift: rows of dense tensors, or
// as good as, with a number of channels that is no multiple of 8, so that row m starts m D mod 8 = s values behind a
// 16-byte boundary, in all tensors alike: a chunk is 16-byte aligned and its first channel is s below a multiple of
// 8, the first and last chunk of a row hold neighbours' values, which read as zero (65536 x 1001, bf16: forward
// 102 us, 139 value by value, backward 107 and 172).  kAny: anything else, value by value.
enum Access { kAny, kVec, kShift };
// The places in a row that hold its channels, counted from its first chunk on: none where there is no row.
// `last`: memory may end behind them.
struct Span {
  int lo, hi;
  bool last;
};
__device__ __forceinline__ int shift_of(long long row, int D) { return (int)(row * D & 7); }

// Chunk r of a thread's channels of a row, as loaded, so that a load can be started ahead of its use.
// Channels that are not there are zero and are not stored.
template <typename T, int A>
struct Raw8 {
  uint4 u[sizeof(T) / 2];
  // kAny: channel i of the chunk.
  static __device__ __forceinline__ int channel(int r, int i) { return (8 * r + i) * blockDim.x + threadIdx.x; }
  static __device__ __forceinline__ int first(int r) { return 8 * (threadIdx.x + r * blockDim.x); }
  __device__ __forceinline__ void load(const T* row, int r, const Span& d) {
    if constexpr (A == kAny) {
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = channel(r, i) < d.hi ? bits_at(row, channel(r, i)) : 0u;
      put(v);
    } else if (A == kVec || first(r) + 8 <= d.hi || !d.last) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i)
        u[i] = first(r) < d.hi ? reinterpret_cast<const uint4*>(row + first(r))[i] : make_uint4(0, 0, 0, 0);
      mask(r, d);
    } else {
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = first(r) + i < d.hi ? bits_at(row, first(r) + i) : 0u;
      put(v);
      mask(r, d);
    }
  }
  // kShift: neighbours' values become zero.
  __device__ __forceinline__ void mask(int r, const Span& d) {
    if (A != kShift || (first(r) >= d.lo && first(r) + 8 <= d.hi)) return;
    uint32_t v[8];
    take(v);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (first(r) + i < d.lo || first(r) + i >= d.hi) v[i] = 0;
    put(v);
  }
  static __device__ __forceinline__ uint32_t bits_at(const T* row, int c) {
    if constexpr (sizeof(T) == 4)
      return __float_as_uint(row[c]);
    else
      return row[c];
  }
  __device__ __forceinline__ void put(const uint32_t (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
      u[0] = make_uint4(v[0], v[1], v[2], v[3]);
      u[sizeof(T) / 2 - 1] = make_uint4(v[4], v[5], v[6], v[7]);
    } else {
      u[0] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
  }
  __device__ __forceinline__ void take(uint32_t (&v)[8]) const {
    const uint4 a = u[0], b = u[sizeof(T) / 2 - 1];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = sizeof(T) == 4 ? w[i] : w[i / 2] >> (16 * (i & 1)) & 0xffffu;
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
  __device__ __forceinline__ void store(T* row, int r, const Span& d) const {
    if (A == kVec ? first(r) < d.hi : A == kShift && first(r) >= d.lo && first(r) + 8 <= d.hi) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(row + first(r))[i] = u[i];
    } else if (A != kVec && (A == kAny || first(r) < d.hi)) {
      uint32_t v[8];
      take(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = A == kAny ? channel(r, i) : first(r) + i;
        if (c < d.lo || c >= d.hi) continue;
        if constexpr (sizeof(T) == 4)
          row[c] = __uint_as_float(v[i]);
        else
          row[c] = (uint16_t)v[i];
      }
    }
  }
};
// The weights of chunk r.  kShift: of two chunks of w, by the row's shift (3000 x 9001, bf16, backward: 109 us; moved
// by powers of two, 121).
template <int A>
__device__ __forceinline__ void load_weight(const float* w, int r, const Span& d, int D, float2 (&f)[4]) {
  if constexpr (A != kShift) {
    Raw8<float, A> u;
    u.load(w, r, Span{0, D, false});
    u.get(f);
  } else {
    float v[16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = Raw8<float, A>::first(r) + 8 * h - 8;
      if (c >= 0 && c + 8 <= D) {
        const float4 a = reinterpret_cast<const float4*>(w + c)[0], b = reinterpret_cast<const float4*>(w + c)[1];
        v[8 * h] = a.x, v[8 * h + 1] = a.y, v[8 * h + 2] = a.z, v[8 * h + 3] = a.w;
        v[8 * h + 4] = b.x, v[8 * h + 5] = b.y, v[8 * h + 6] = b.z, v[8 * h + 7] = b.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * h + i] = c + i >= 0 && c + i < D ? w[c + i] : 0.f;
      }
    }
    auto pick = [&](auto shift) {
      constexpr int from = 8 - decltype(shift)::value;
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = make_float2(v[from + 2 * i], v[from + 2 * i + 1]);
    };
    switch (d.lo) {
      case 1: pick(Int<1>{}); break;
      case 2: pick(Int<2>{}); break;
      case 3: pick(Int<3>{}); break;
      case 4: pick(Int<4>{}); break;
      case 5: pick(Int<5>{}); break;
      case 6: pick(Int<6>{}); break;
      case 7: pick(Int<7>{}); break;
      default: pick(Int<0>{});
    }
  }
}

__device__ __forceinline__ float across(float x, int lanes) { return x + __shfl_xor_sync(~0u, x, lanes); }
__device__ __forceinline__ float2 across(float2 x, int lanes) {
  return add2(x, make_float2(__shfl_xor_sync(~0u, x.x, lanes), __shfl_xor_sync(~0u, x.y, lanes)));
}
// Sum over the threads of a row, for each of them: of one value or two.  `turn` (0, 1, 0, ...) chooses the
// scratch, so that one barrier a sum is enough.
template <typename V>
__device__ __forceinline__ V row_sum(V s, int turn) {
  __shared__ V part[2][16];
  if (blockDim.x > 16) s = across(s, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) s = across(s, o);
  if (blockDim.x > 32) {  // and then a row has the block for itself
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = s;
    __syncthreads();
    if constexpr (sizeof(V) == 8) {  // shorter: no shuffles in a row (16384 x 8192: 161 us instead of 172)
      s = part[turn][0];
      for (int w = 1; w < warps; ++w) s = add2(s, part[turn][w]);
    } else {  // fewer instructions
      const int w = threadIdx.x & 15;
      s = w < warps ? part[turn][w] : V{};
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) s = across(s, o);
    }
  }
  return s;
}

// The larger of two |values|, NaN if either is.
__device__ __forceinline__ float larger(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// Chunk r of a row in 8 bits: 16 threads to a scale, TAIL where the row's last chunk may be shorter.  v holds h w; the result is v inv.  The largest |v inv| is
// the largest |v| times inv, rounding being monotonic, and the scale's inverse, a power of two, goes with inv.
template <bool TAIL>
__device__ __forceinline__ void store_fp8(const float2 (&v)[4], float inv, int r, int D, uint8_t* q, uint8_t* scales) {
  float top = larger(larger(larger(v[0].x, v[0].y), larger(v[1].x, v[1].y)),
                     larger(larger(v[2].x, v[2].y), larger(v[3].x, v[3].y)));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) top = larger(top, __shfl_xor_sync(~0u, top, o));
  const uint32_t e = scale_exponent(__float_as_uint(top * inv) & 0x7fffffffu);
  const float2 by = pair(inverse_scale(e));
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = mul2(mul2(v[i], pair(inv)), by);
    b[i] = pack_e4m3x2(y.x, y.y);
  }
  const int c = 8 * (threadIdx.x + r * blockDim.x);
  if (c >= D) return;
  if (c % kScaleBlock == 0) scales[c / kScaleBlock] = (uint8_t)e;
  if (!TAIL || c + 8 <= D) {
    *reinterpret_cast<uint2*>(q + c) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (c + i < D) q[c + i] = (uint8_t)(b[i / 2] >> (8 * (i & 1)));
  }
}
// kShift in 8 bits: a row's values pass through shared memory, as scales and q follow the row.  Value c is at c +
// c / 32, so that threads eight apart meet different banks (65536 x 1001, bf16 with residual: 108 us; value by value
// 196).
__host__ __device__ constexpr int place_of(int c) { return c + c / 32; }
// |values| as bits, which order them and put NaN above all.
__device__ __forceinline__ uint32_t bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// A row in 8 bits, kAny: a row has one warp, and the 128 channels of a scale are four values of each lane,
// or a multiple of 128 threads, and they are one value of each thread of four warps.
template <int R>
__device__ __forceinline__ void store_fp8_any(const float2 (&v)[R][4], int D, uint8_t* q, uint8_t* scales) {
  __shared__ uint32_t tops[8 * R][16];
  const int warp = threadIdx.x >> 5;
  const float* value = &v[0][0].x;
  const bool alone = blockDim.x == 32;
  if (!alone) {
#pragma unroll
    for (int i = 0; i < 8 * R; ++i) {
      const uint32_t top = __reduce_max_sync(~0u, bits(value[i]));
      if ((threadIdx.x & 31) == 0) tops[i][warp] = top;
    }
    __syncthreads();
  }
  uint32_t e = 0;
#pragma unroll
  for (int i = 0; i < 8 * R; ++i) {
    if (!alone) {
      const uint32_t* t = &tops[i][warp & ~3];
      e = scale_exponent(max(max(t[0], t[1]), max(t[2], t[3])));
    } else if (i % 4 == 0) {
      e = scale_exponent(__reduce_max_sync(
          ~0u, max(max(bits(value[i]), bits(value[i + 1])), max(bits(value[i + 2]), bits(value[i + 3])))));
    }
    const int c = i * blockDim.x + threadIdx.x;
    if (c < D) {
      if (c % kScaleBlock == 0) scales[c / kScaleBlock] = (uint8_t)e;
      q[c] = (uint8_t)pack_e4m3x2(value[i] * inverse_scale(e), 0.f);
    }
  }
}

// Two blocks of 512 threads to an SM where a thread has one chunk (or two, not kAny): left alone, the compiler takes
// 128 registers for a chunk of eight separate channels.
template <typename T, bool FP8, int A, int R>
__global__ void __launch_bounds__(512, R == 1 || (A != kAny && R == 2) ? 2 : 1)
    add_rmsnorm_kernel(AddNormProblem p, uint16_t* __restrict__ out, uint8_t* __restrict__ q, long long q_row,
                       uint8_t* __restrict__ scales) {
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const int lo = A == kShift ? shift_of(row, p.D) : 0;
  const Span d{lo, row < p.rows ? lo + p.D : 0, row + 1 >= p.rows};  // behind the last row there are no channels
  const T* stream = static_cast<const T*>(p.stream) + row * p.stream_row - lo;
  const uint16_t* x = p.x ? p.x + row * p.x_row - lo : nullptr;
  extern __shared__ float turned[];
  [[maybe_unused]] float* turn = turned + threadIdx.y * place_of(p.D + 31);
  float2 h[R][4], s = pair(0.f);
  Raw8<T, A> a[R];
  Raw8<uint16_t, A> b[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    a[r].load(stream, r, d);
    if (x) b[r].load(x, r, d);
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
    if (p.h) a[r].store(static_cast<T*>(p.h) + row * p.D - lo, r, d);
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fma2(h[r][i], h[r][i], s);
    if constexpr (FP8 && A == kShift) {
      const float* value = &h[r][0].x;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = Raw8<T, A>::first(r) + i - lo;
        if (c >= 0 && c < p.D) turn[place_of(c)] = value[i];
      }
    }
  }
  if (FP8 && A == kShift) __syncwarp();  // wider rows pass the sum's barrier
  const float inv = rsqrtf(row_sum(s.x + s.y, 0) * (1.f / (float)p.D) + p.eps);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float2 w[4];
    if constexpr (FP8 && A == kShift) {
      const int c = Raw8<T, A>::first(r);
      float* value = &h[r][0].x;
#pragma unroll
      for (int i = 0; i < 8; ++i) value[i] = c + i < p.D && d.hi > 0 ? turn[place_of(c) + i] : 0.f;
      load_weight<A>(p.w, r, Span{0, p.D, false}, p.D, w);
    } else {
      load_weight<A>(p.w, r, d, p.D, w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) h[r][i] = mul2(h[r][i], w[i]);
    if constexpr (!FP8 || A == kAny)  // store_fp8 does it itself
#pragma unroll
      for (int i = 0; i < 4; ++i) h[r][i] = mul2(h[r][i], pair(inv));
    if constexpr (FP8 && A != kAny) {
      store_fp8<A == kShift>(h[r], inv, r, d.hi > 0 ? p.D : 0, q + row * q_row, scales + row * scale_blocks(p.D));
    } else if constexpr (!FP8) {
      Raw8<uint16_t, A> o;
      o.set(h[r]);
      o.store(out + row * p.D - lo, r, d);
    }
  }
  if constexpr (FP8 && A == kAny) store_fp8_any<R>(h, d.hi, q + row * q_row, scales + row * scale_blocks(p.D));
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
template <bool SECTORS>
__device__ __forceinline__ void copy16(uint32_t to, const void* from, int bytes) {  // and zeros behind them
  if constexpr (SECTORS)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
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
template <typename T, int A, int R, bool MULTI>
struct RowStream {
  static constexpr int kRows = kAhead<T, R>, kParts = sizeof(T) / 2;  // 16-byte pieces of 8 values
  const AddNormBackwardProblem& p;
  uint4* own;  // [kRows][kParts + 1 + kParts][R][threads of the block]
  const int lo;  // a thread's rows all have the same shift
  int at = 0, to = 0;
  Raw8<T, A> hr[R], er[R];
  Raw8<uint16_t, A> dr[R];

  __device__ __forceinline__ RowStream(const AddNormBackwardProblem& p_, int lo_, uint4* smem)
      : p(p_), own(smem + (MULTI ? threadIdx.y * blockDim.x : 0) + threadIdx.x), lo(lo_) {}
  __device__ __forceinline__ Span span(long long row) const {
    return Span{lo, row < p.rows ? lo + p.D : 0, row + 1 >= p.rows};
  }
  __device__ __forceinline__ uint4* slot(int stage, int part, int r) const {
    return own + ((stage * (2 * kParts + 1) + part) * R + r) * (blockDim.x * (MULTI ? blockDim.y : 1));
  }
  __device__ __forceinline__ void start(long long row) {
    if (row < p.rows) {
      const Span s = span(row);
      const T *h = static_cast<const T*>(p.h) + row * p.D - lo, *e = static_cast<const T*>(p.dh) + row * p.D - lo;
      const uint16_t* d = p.dout + row * p.D - lo;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if constexpr (A != kAny) {
          const int c = Raw8<T, A>::first(r);
          // Part k of `parts` of eight values: of the last row only what is there.
          auto copy = [&](auto sectors, int part, const void* from, int k, int parts) {
            const uint32_t at = smem_u32(slot(to, part, r));
            const uint4* v = static_cast<const uint4*>(from) + k;
            const int each = 8 / parts;
            if (A == kShift && s.last)
              copy16<decltype(sectors)::value>(at, v, max(0, min(each, s.hi - c - k * each)) * (16 / each));
            else
              copy16<decltype(sectors)::value>(at, v);
          };
          if (c < s.hi) {
#pragma unroll
            for (int k = 0; k < kParts; ++k) copy(Int<kParts == 2>{}, k, h + c, k, kParts);
            copy(Int<false>{}, kParts, d + c, 0, 1);
            if (p.dh)
#pragma unroll
              for (int k = 0; k < kParts; ++k) copy(Int<kParts == 2>{}, kParts + 1 + k, e + c, k, kParts);
          }
        } else {
          hr[r].load(h, r, s);
          dr[r].load(d, r, s);
          if (p.dh) er[r].load(e, r, s);
        }
      }
    }
    if constexpr (A != kAny) {
      copies_commit();
      to = to + 1 == kRows ? 0 : to + 1;
    }
  }
  __device__ __forceinline__ void begin(long long row, long long step) {
#pragma unroll
    for (int i = 0; i < (A != kAny ? kRows - 1 : kParts / kParts); ++i) start(row + i * step);
  }
  // dh of the row at hand is taken before the sums where there is room to hold it across them (65536 x 2048
  // float32: 317 us, 364 where it is taken after them; 4000 x 16384 bf16: 215 and 124).
  static constexpr bool kEarly = A != kAny && R <= 2;
  // h, dout and, if early, dh of `row`, zeros where its span has no channels; a later row starts.
  __device__ __forceinline__ void next(long long row, const Span& s, long long step, float2 (&h)[R][4],
                                       float2 (&d)[R][4], float2 (&e)[R][4]) {
    if constexpr (A != kAny) {
      start(row + (kRows - 1) * step);
      copies_wait<kRows - 1>();
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int i = 0; i < 4; ++i) h[r][i] = d[r][i] = e[r][i] = pair(0.f);
      if (A != kAny ? Raw8<T, A>::first(r) < s.hi : s.hi > 0) {
        if constexpr (A != kAny) {
#pragma unroll
          for (int k = 0; k < kParts; ++k) hr[r].u[k] = *slot(at, k, r);
          dr[r].u[0] = *slot(at, kParts, r);
          if (kEarly && p.dh)
#pragma unroll
            for (int k = 0; k < kParts; ++k) er[r].u[k] = *slot(at, kParts + 1 + k, r);
          hr[r].mask(r, s), dr[r].mask(r, s);  // of dh, neighbours' values change nothing
        }
        hr[r].get(h[r]);
        dr[r].get(d[r]);
        if (kEarly && p.dh) er[r].get(e[r]);
      }
    }
  }
  // dh of chunk r, where it is late.
  __device__ __forceinline__ void late(int r, const Span& s, float2 (&e)[4]) {
    if (kEarly || !p.dh || (A != kAny ? Raw8<T, A>::first(r) >= s.hi : s.hi == 0)) return;
    if constexpr (A != kAny)
#pragma unroll
      for (int k = 0; k < kParts; ++k) er[r].u[k] = *slot(at, kParts + 1 + k, r);
    er[r].get(e);
  }
  __device__ __forceinline__ void done(long long row, long long step) {
    if constexpr (A != kAny)
      at = at + 1 == kRows ? 0 : at + 1;
    else
      start(row + step);
  }
};

// Block b takes rows b, + blocks, ... (MULTI: blockDim.y of them at once); its channels' part of dw adds up in
// registers and goes to row b of `part`.
template <typename T, int A, int R, bool MULTI>
__global__ void __launch_bounds__(512, R == 1 ? 2 : 1)
    add_rmsnorm_backward_kernel(AddNormBackwardProblem p, float* __restrict__ part) {
  extern __shared__ uint4 ring[];
  const float inv_d = 1.f / (float)p.D;
  constexpr bool kKeep = R <= 2;  // the weight stays in registers where there is room for it
  float2 dw[R][4], kept[kKeep ? R : 1][4];
  const int at_once = MULTI ? blockDim.y : 1;
  const long long step = (long long)gridDim.x * at_once;
  long long row = (long long)blockIdx.x * at_once + (MULTI ? threadIdx.y : 0);
  // The shift of all of a thread's rows: more than one only where the grid is a multiple of 8.
  const int lo = A == kShift ? shift_of(row, p.D) : 0;
  auto weight = [&](int r, float2(&w)[4]) { load_weight<A>(p.w, r, Span{lo, lo + p.D, false}, p.D, w); };
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if constexpr (kKeep) weight(r, kept[r]);
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[r][i] = pair(0.f);
  }
  RowStream<T, A, R, MULTI> rows(p, lo, ring);
  rows.begin(row, step);
  int turn = 0;
  // All threads of a block go round equally often; behind the last row there are no channels.
  for (long long first = (long long)blockIdx.x * at_once; first < p.rows; first += step, row += step, turn ^= 1) {
    const Span span = rows.span(row);
    float2 h[R][4], d[R][4], s1 = pair(0.f), s2 = pair(0.f);
    float2 e[R][4];
    rows.next(row, span, step, h, d, e);
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
    const float2 sum = row_sum(make_float2(s1.x + s1.y, s2.x + s2.y), turn);
    const float inv = !MULTI || span.hi > 0 ? rsqrtf(sum.x * inv_d + p.eps) : 0.f;
    // In this order: inv^3 leaves float32 where |h| is above 1e13 or below 1e-13.
    const float2 iv = pair(inv), back = pair(-(sum.y * inv_d * inv) * inv * inv);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 o[4], w[4];
      rows.late(r, span, e[r]);
      if constexpr (!kKeep) weight(r, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dw[r][i] = fma2(d[r][i], mul2(h[r][i], iv), dw[r][i]);
        o[i] = add2(fma2(h[r][i], back, mul2(mul2(d[r][i], kKeep ? kept[kKeep ? r : 0][i] : w[i]), iv)), e[r][i]);
      }
      if (p.dx) {
        Raw8<uint16_t, A> u;
        u.set(o);
        u.store(p.dx + row * p.D - lo, r, span);
      }
      if (p.dresidual) {
        Raw8<T, A> u;
        u.set(o);
        u.store(static_cast<T*>(p.dresidual) + row * p.D - lo, r, span);
      }
    }
    rows.done(row, step);
  }
  float* to = part + (long long)blockIdx.x * p.D;
  if (MULTI) {  // the block's rows at once add up first, in the rows' place
    copies_wait<0>();
    __syncthreads();
    to = reinterpret_cast<float*>(ring) + threadIdx.y * p.D;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if constexpr (A == kShift) {
      const float* value = &dw[r][0].x;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = Raw8<float, A>::first(r) + i - lo;
        if (c >= 0 && c < p.D) to[c] = value[i];
      }
    } else {
      Raw8<float, A> u;
      u.set(dw[r]);
      u.store(to, r, Span{0, p.D, false});
    }
  }
  if (MULTI) {
    __syncthreads();
    for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < p.D; c += blockDim.x * blockDim.y) {
      float s = 0.f;
      for (int y = 0; y < blockDim.y; ++y) s += reinterpret_cast<const float*>(ring)[y * p.D + c];
      part[(long long)blockIdx.x * p.D + c] = s;
    }
  }
}

// How rows are spread: chunks and threads per row, rows per block.
struct Spread {
  int R, threads, rows;
  dim3 block() const { return dim3(threads, rows); }
};
// Threads of a row for R chunks each: half a warp, whole warps, or (8 bits, kAny) a warp or four at a time.
int threads_for(int D, int R, Access a, bool fp8) {
  const int n = ((D + (a == kShift ? 7 : 0) + 7) / 8 + R - 1) / R;
  if (a != kAny && n <= 16) return 16;
  const int whole = a == kAny && fp8 && n > 32 ? 128 : 32;
  return (n + whole - 1) / whole * whole;
}
// With `least` chunks a thread, or more where a row would have more than 512 threads.
Spread spread_of(int D, int least, Access a, bool fp8) {
  int R = least;
  while (threads_for(D, R, a, fp8) > 512) R *= 2;
  const int threads = threads_for(D, R, a, fp8);
  return Spread{R, threads, threads <= 32 ? 256 / threads : 1};
}

template <typename F>
cudaError_t with_chunks(int R, F f) {
  return R == 1 ? f(Int<1>{}) : R == 2 ? f(Int<2>{}) : f(Int<4>{});
}

// Chunks a thread of many rows (few are spread as wide as they go): two (65536 x 2048 bf16 with residual: 153 us,
// with one 169, with four 158), of which a thread's loads are on their way together.  Four where they are of two
// bytes a channel, or of four and the result of one, and rows are long: less of a block's time is then spent on
// sums (16384 x 4096 bf16 without residual: in 8 bits 47 us instead of 54, in bf16 43 instead of 47; with residual,
// in 8 bits, 71.7 instead of 73.1).  One where 16 threads hold the row so (498379 x 96 in 8 bits: 47 instead of 72).
int chunks_of(const AddNormProblem& p, Access a, bool fp8) {
  if (a == kAny || p.D + (a == kShift ? 7 : 0) <= 16 * 8) return 1;
  const int read = (p.stream_f32 ? 4 : 2) + (p.x ? 2 : 0);
  const bool four = fp8 ? p.D >= (read == 2 ? 512 : 4096) && read <= 4 : p.D >= 2048 && read == 2;
  return a == kVec && four ? 4 : 2;
}

template <typename T, bool FP8, Access A>
cudaError_t forward(const AddNormProblem& p, uint16_t* out, uint8_t* q, long long q_row, uint8_t* scales,
                    cudaStream_t stream) {
  const bool many = p.rows >= 152 * 16;
  Spread s = spread_of(p.D, many ? chunks_of(p, A, FP8) : 1, A, FP8);
  if (!many) s.rows = s.threads < 32 ? 2 : 1;
  return with_chunks(s.R, [&](auto r) {
    const long long blocks = (p.rows + s.rows - 1) / s.rows;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;  // more than a terabyte
    auto* kernel = add_rmsnorm_kernel<T, FP8, A, decltype(r)::value>;
    const int bytes = FP8 && A == kShift ? s.rows * place_of(p.D + 31) * (int)sizeof(float) : 0;
    if constexpr (FP8 && A == kShift) {
      // At every launch, as the attribute belongs to the current device, and for the widest row, whatever this call's
      // is: another thread's call may be between its attribute and its launch.  (Several rows a block: under 18 KB.)
      constexpr int kMost = place_of(kNormMaxRow + 31) * (int)sizeof(float);
      const cudaError_t attr = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
      if (attr != cudaSuccess) return attr;
    }
    kernel<<<(unsigned)blocks, s.block(), bytes, stream>>>(p, out, q, q_row, scales);
    return cudaGetLastError();
  });
}

// Whether rows of D values can be read as kShift: a chunk may reach up to 7 values into the next row.
bool shift_ok(int D) { return D >= 8 && D + 7 <= kNormMaxRow; }

// `rest`: whether what is particular to the call starts on 16 bytes.
Access access_of(const AddNormProblem& p, bool rest) {
  const size_t size = p.stream_f32 ? 4 : 2;
  if (!rest || !aligned_to(p.w, 16) || !aligned_to(p.h, 16) || !aligned_to(p.stream, 16) || !aligned_to(p.x, 16))
    return kAny;
  if (p.D % 8 == 0) return p.stream_row * size % 16 == 0 && (!p.x || p.x_row % 8 == 0) ? kVec : kAny;
  auto alike = [&](long long row) { return row >= p.D && (row - p.D) % 8 == 0; };
  return shift_ok(p.D) && alike(p.stream_row) && (!p.x || alike(p.x_row)) ? kShift : kAny;
}

template <typename T, bool FP8>
cudaError_t dispatch(const AddNormProblem& p, Access a, uint16_t* out, uint8_t* q, long long q_row, uint8_t* scales,
                     cudaStream_t stream) {
  if (a == kVec) return forward<T, FP8, kVec>(p, out, q, q_row, scales, stream);
  if (a == kShift) return forward<T, FP8, kShift>(p, out, q, q_row, scales, stream);
  return forward<T, FP8, kAny>(p, out, q, q_row, scales, stream);
}

// The backward's spread (several rows a block only with a chunk per thread), and its blocks, which are the rows of
// its sums: 1024 threads for every SM.
Spread backward_spread(int D, Access a) { return spread_of(D, 1, a, false); }
int backward_blocks(long long rows, int D, Access a) {
  const Spread s = backward_spread(D, a);
  const long long most = 152LL * (1024 / (s.threads * s.rows)), all = (rows + s.rows - 1) / s.rows;
  return (int)(all < most ? (all > 0 ? all : 1) : most);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const AddNormProblem& p, uint16_t* out, cudaStream_t stream) {
  const Access a = access_of(p, aligned_to(out, 16));
  return p.stream_f32 ? dispatch<float, false>(p, a, out, nullptr, 0, nullptr, stream)
                      : dispatch<uint16_t, false>(p, a, out, nullptr, 0, nullptr, stream);
}
cudaError_t launch_add_rmsnorm_fp8(const AddNormProblem& p, uint8_t* q, long long q_row, uint8_t* scales,
                                   cudaStream_t stream) {
  const Access a = access_of(p, true);
  return p.stream_f32 ? dispatch<float, true>(p, a, nullptr, q, q_row, scales, stream)
                      : dispatch<uint16_t, true>(p, a, nullptr, q, q_row, scales, stream);
}

size_t add_rmsnorm_backward_workspace_floats(long long rows, int D) {
  const int a = backward_blocks(rows, D, kAny);
  const int b = D % 8 == 0 ? backward_blocks(rows, D, kVec) : shift_ok(D) ? backward_blocks(rows, D, kShift) : 0;
  return (size_t)(a > b ? a : b) * D;
}

cudaError_t launch_add_rmsnorm_backward(const AddNormBackwardProblem& p, cudaStream_t stream) {
  if (p.rows == 0) return cudaMemsetAsync(p.dw, 0, sizeof(float) * p.D, stream);
  const bool aligned = aligned_to(p.w, 16) && aligned_to(p.h, 16) && aligned_to(p.dout, 16) && aligned_to(p.dh, 16) &&
                       aligned_to(p.dx, 16) && aligned_to(p.dresidual, 16);
  const Access a = !aligned ? kAny : p.D % 8 == 0 ? kVec : shift_ok(p.D) ? kShift : kAny;
  const int blocks = backward_blocks(p.rows, p.D, a);
  const Spread s = backward_spread(p.D, a);
  const cudaError_t err = with_chunks(s.R, [&](auto r) {
    constexpr int R = decltype(r)::value;
    auto go = [&](auto kernel) {
      const int each = p.stream_f32 ? kRingPerThread<float, R> : kRingPerThread<uint16_t, R>;
      constexpr int kMost = 512 * (kRingPerThread<float, R> > kRingPerThread<uint16_t, R> ? kRingPerThread<float, R>
                                                                                          : kRingPerThread<uint16_t, R>);
      const int ring = a != kAny ? s.threads * s.rows * each : 0;
      const int sums = s.rows > 1 ? s.rows * p.D * 4 : 0, bytes = ring > sums ? ring : sums;
      // At every launch, as the attribute belongs to the current device, and for the largest block, whatever this call's
      // is: another thread's call may be between its attribute and its launch.  (Sums of several rows: 8 KB at most.)
      const cudaError_t attr = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
      if (attr != cudaSuccess) return attr;
      kernel<<<blocks, s.block(), bytes, stream>>>(p, p.ws);
      return cudaGetLastError();
    };
    auto with = [&](auto access) {
      constexpr int A = decltype(access)::value;
      if constexpr (R == 1)
        if (s.rows > 1)
          return p.stream_f32 ? go(add_rmsnorm_backward_kernel<float, A, 1, true>)
                              : go(add_rmsnorm_backward_kernel<uint16_t, A, 1, true>);
      return p.stream_f32 ? go(add_rmsnorm_backward_kernel<float, A, R, false>)
                          : go(add_rmsnorm_backward_kernel<uint16_t, A, R, false>);
    };
    return a == kVec ? with(Int<kVec>{}) : a == kShift ? with(Int<kShift>{}) : with(Int<kAny>{});
  });
  if (err != cudaSuccess) return err;
  return launch_sum_rows(p.ws, p.dw, nullptr, blocks, p.D, p.D, p.D, stream);
}

}  // namespace m2rnn
