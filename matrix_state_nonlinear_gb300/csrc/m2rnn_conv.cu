// m2rnn_conv.cu — the short causal convolution (4 taps, depthwise, SiLU) with a carried window,
// and its backward pass.
//
//   pre[t] = bias + sum_j w[j] X[t-3+j],  out = pre sigmoid(pre),  X = window then x
//   dpre[t] = dout[t] sigma (1 + pre (1 - sigma))
//   dX[t] = sum_j w[j] dpre[t+3-j],  dw[j] = sum_{b,t} dpre[t] X[t-3+j],  dbias = sum dpre
//
// Memory-bound: the forward reads and writes every element once (4 bytes an element), the
// backward reads two and writes one (6 bytes).  A thread owns four neighbouring channels (8-byte
// accesses, arithmetic in pairs) over a stretch of tokens; eight (four) tokens are loaded at once
// and joined to the last three in registers, so that enough bytes are in flight and the window
// moves once per group of tokens.  The three tokens that stretches share are re-read, from L2.
// Measured, 8 x 8192 tokens of 2304 channels: forward 95 us (6.3 TB/s, 93 % of a copy; stretches of 64
// tokens, of 128 98 us), backward (of 128; of 64 175 us and 12 us for the sums) 169 us
// (5.4 TB/s; with loads to registers, three blocks an SM, 202 us) and 8 us for the sums.
#include "m2rnn_ssm.h"
#include "ptx_util.cuh"

namespace m2rnn {
namespace {

constexpr int kTaps = 4;
constexpr int kHist = kTaps - 1;
constexpr int kThreads = 128;

// VEC channels (4 or 1) of one token: raw, and as float pairs (one pair of which half is used).
template <int VEC>
struct Chan;
template <>
struct Chan<4> {
  using Raw = uint2;
  static constexpr int P = 2;
  __device__ static void unpack(uint2 u, float2 (&f)[2]) {
    f[0] = bf16x2_to_float2(u.x), f[1] = bf16x2_to_float2(u.y);
  }
  __device__ static uint2 pack(const float2 (&f)[2]) {
    return make_uint2(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y));
  }
};
template <>
struct Chan<1> {
  using Raw = uint16_t;
  static constexpr int P = 1;
  __device__ static void unpack(uint16_t u, float2 (&f)[1]) { f[0] = make_float2(bf16_to_f(u), 0.f); }
  __device__ static uint16_t pack(const float2 (&f)[1]) { return f_to_bf16(f[0].x); }
};

// A thread's channels: taps as pairs, bias.
template <int VEC>
struct Taps {
  static constexpr int P = Chan<VEC>::P;
  float2 w[kTaps][P], b[P];
  __device__ __forceinline__ void load(const float* wp, const float* bias, int c0) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(wp + (size_t)(c0 + 2 * i) * kTaps);
      const float4 y = VEC > 1 ? *reinterpret_cast<const float4*>(wp + (size_t)(c0 + 2 * i + 1) * kTaps) : x;
      w[0][i] = make_float2(x.x, y.x), w[1][i] = make_float2(x.y, y.y);
      w[2][i] = make_float2(x.z, y.z), w[3][i] = make_float2(x.w, y.w);
      b[i] = bias ? make_float2(bias[c0 + 2 * i], VEC > 1 ? bias[c0 + 2 * i + 1] : 0.f) : make_float2(0.f, 0.f);
    }
  }
};

// X[t] of one batch row: the window for t in [-3, -1], x after that; zeros past the sequence.
template <int VEC>
__device__ __forceinline__ typename Chan<VEC>::Raw load_x(const uint16_t* xb, const uint16_t* win, long long x_token,
                                                          int C, int T, int t) {
  using Raw = typename Chan<VEC>::Raw;
  const uint16_t* p = t >= 0 ? xb + t * x_token : win + (long long)(t + kHist) * C;
  return t < T && (t >= 0 || win) ? *reinterpret_cast<const Raw*>(p) : Raw{};
}

// Forward: one thread, VEC channels, `span` tokens of one batch row.  The thread of the first
// stretch also writes the window after x: it alone reads window_in, so that the two may be the
// same memory.
template <int VEC>
__global__ void __launch_bounds__(kThreads)
    conv_window_kernel(ConvProblem p, uint16_t* __restrict__ out, uint16_t* window_out, int span,
                       int groups, int stretches) {
  using Ch = Chan<VEC>;
  using Raw = typename Ch::Raw;
  constexpr int P = Ch::P, U = 8;
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int c0 = VEC * (int)(id % groups);
  const int stretch = (int)(id / groups % stretches);
  const long long b = id / groups / stretches;
  if (b >= p.B) return;
  const uint16_t* xb = p.x + b * p.sx.batch + c0;
  const uint16_t* win = p.window_in ? p.window_in + b * kHist * p.C + c0 : nullptr;
  const int t0 = stretch * span, t1 = min(p.T, t0 + span);
  uint16_t* ob = out + (b * p.T + t0) * p.C + c0;
  float2 x[U + kHist][P];  // X[t - 3], ...
#pragma unroll
  for (int j = 0; j < kHist; ++j) Ch::unpack(load_x<VEC>(xb, win, p.sx.token, p.C, p.T, t0 - kHist + j), x[j]);
  if (stretch == 0 && window_out) {
    Raw f[kHist];
#pragma unroll
    for (int j = 0; j < kHist; ++j) f[j] = load_x<VEC>(xb, win, p.sx.token, p.C, p.T, p.T - kHist + j);
#pragma unroll
    for (int j = 0; j < kHist; ++j) *reinterpret_cast<Raw*>(window_out + (b * kHist + j) * p.C + c0) = f[j];
  }
  Taps<VEC> w;
  w.load(p.w, p.bias, c0);
  Raw raw[U];
  const uint16_t* next = xb + t0 * p.sx.token;
  auto fetch = [&](int t) {
#pragma unroll
    for (int u = 0; u < U; ++u, next += p.sx.token)
      if (t + u < t1) raw[u] = *reinterpret_cast<const Raw*>(next);
  };
  fetch(t0);
  for (int t = t0; t < t1; t += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) Ch::unpack(raw[u], x[kHist + u]);
    fetch(t + U);  // while these are computed
#pragma unroll
    for (int u = 0; u < U; ++u, ob += p.C) {
      if (t + u >= t1) break;
      float2 o[P];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float2 s = fma2(w.w[0][i], x[u][i], w.b[i]);
        s = fma2(w.w[1][i], x[u + 1][i], s);
        s = fma2(w.w[2][i], x[u + 2][i], s);
        s = fma2(w.w[3][i], x[u + 3][i], s);
        o[i] = mul2(s, sigmoid2(s));
      }
      *reinterpret_cast<Raw*>(ob) = Ch::pack(o);
    }
#pragma unroll
    for (int j = 0; j < kHist; ++j)
#pragma unroll
      for (int i = 0; i < P; ++i) x[j][i] = x[U + j][i];
  }
}

// Eight bytes to shared memory, asynchronously; zeros without `in`.
__device__ __forceinline__ void copy8(void* dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 8 : 0)
               : "memory");
}

template <bool V>
struct Flag {
  static constexpr bool value = V;
};

// Backward: one thread, VEC channels, `span` tokens of one batch row.  dX[t] needs dpre up to
// t + 3, so the thread runs three tokens past its stretch; only its own tokens enter dw, dbias.
// The partial sums of each (batch row, stretch) go to `part` [rows][C][5].
template <int VEC>
__global__ void __launch_bounds__(kThreads, 4)
    conv_backward_kernel(ConvProblem p, const uint16_t* __restrict__ dout,
                         uint16_t* __restrict__ dx, uint16_t* __restrict__ dwindow,
                         float* __restrict__ part, int span, int groups, int stretches) {
  using Ch = Chan<VEC>;
  using Raw = typename Ch::Raw;
  constexpr int P = Ch::P, U = 4;
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int c0 = VEC * (int)(id % groups);
  const int stretch = (int)(id / groups % stretches);
  const long long b = id / groups / stretches;
  if (b >= p.B) return;
  const uint16_t* xb = p.x + b * p.sx.batch + c0;
  const uint16_t* win = p.window_in ? p.window_in + b * kHist * p.C + c0 : nullptr;
  const int t0 = stretch * span, t1 = min(p.T, t0 + span);
  const float2 zero = make_float2(0.f, 0.f);
  float2 x[U + kHist][P], e[U + kHist][P];  // X[t - 3] ..., dpre[t - 3] ... (zero before the stretch)
  float2 dw[kTaps][P], db[P];
#pragma unroll
  for (int j = 0; j < kHist; ++j) {
    Ch::unpack(load_x<VEC>(xb, win, p.sx.token, p.C, p.T, t0 - kHist + j), x[j]);
#pragma unroll
    for (int i = 0; i < P; ++i) e[j][i] = zero;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    db[i] = zero;
#pragma unroll
    for (int j = 0; j < kTaps; ++j) dw[j][i] = zero;
  }
  Taps<VEC> w;
  w.load(p.w, p.bias, c0);
  const int most = min(p.T, t1 + kHist);
  const uint16_t *nx = xb + t0 * p.sx.token, *ng = dout + (b * p.T + t0) * p.C + c0;
  uint16_t* dxt = dx + (b * p.T + t0 - kHist) * p.C + c0;
  // Loads ahead of their use: four channels by asynchronous copies to the thread's own slots of
  // shared memory, three groups of tokens ahead (no other thread reads them, so nothing but the
  // copies themselves is waited for); one channel to registers, one group ahead.
  constexpr int S = VEC == 4 ? 4 : 1, kAhead = VEC == 4 ? S - 1 : 1;
  __shared__ Raw slots[VEC == 4 ? S : 1][U][2][VEC == 4 ? kThreads : 1];
  Raw xr[U], gr[U];
  int head = 0, tail = 0;
  auto fetch = [&](int t) {
#pragma unroll
    for (int u = 0; u < U; ++u, nx += p.sx.token, ng += p.C) {
      const bool in = t + u < most;
      if constexpr (VEC == 4) {
        copy8(&slots[head][u][0][threadIdx.x], in ? nx : xb, in);
        copy8(&slots[head][u][1][threadIdx.x], in ? ng : dout, in);
      } else if (in) {
        xr[u] = *reinterpret_cast<const Raw*>(nx);
        gr[u] = *reinterpret_cast<const Raw*>(ng);
      } else {
        xr[u] = gr[u] = Raw{};
      }
    }
    if constexpr (VEC == 4) {
      asm volatile("cp.async.commit_group;" ::: "memory");
      head = (head + 1) % S;
    }
  };
  auto take = [&]() {
    if constexpr (VEC == 4) {
      asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
#pragma unroll
      for (int u = 0; u < U; ++u) xr[u] = slots[tail][u][0][threadIdx.x], gr[u] = slots[tail][u][1][threadIdx.x];
      tail = (tail + 1) % S;
    }
  };
  // Tokens t .. t + 3; token t + u completes dX[t + u - 3].  The stretch's own groups (a stretch is
  // a multiple of four tokens, but for the sequence's end, past which dout and so dpre is zero)
  // enter dw and dbias, the one after them does not.
  auto group = [&](int t, auto own) {
    float2 g[U][P];
    take();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Ch::unpack(xr[u], x[kHist + u]);
      Ch::unpack(gr[u], g[u]);
    }
    if (own.value) fetch(t + kAhead * U);  // while these are computed
#pragma unroll
    for (int u = 0; u < U; ++u, dxt += p.C) {
      float2 o[P];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float2 s = fma2(w.w[0][i], x[u][i], w.b[i]);
        s = fma2(w.w[1][i], x[u + 1][i], s);
        s = fma2(w.w[2][i], x[u + 2][i], s);
        s = fma2(w.w[3][i], x[u + 3][i], s);
        const float2 sig = sigmoid2(s), one = make_float2(1.f, 1.f);
        // sigma (1 + s (1 - sigma)); s kept finite where sigma is 0
        s = make_float2(fmaxf(s.x, -1e4f), fmaxf(s.y, -1e4f));
        const float2 d = mul2(g[u][i], mul2(sig, fma2(s, sub2(one, sig), one)));
        if (own.value) {
          db[i] = add2(db[i], d);
          dw[0][i] = fma2(d, x[u][i], dw[0][i]);
          dw[1][i] = fma2(d, x[u + 1][i], dw[1][i]);
          dw[2][i] = fma2(d, x[u + 2][i], dw[2][i]);
          dw[3][i] = fma2(d, x[u + 3][i], dw[3][i]);
        }
        e[kHist + u][i] = d;
        o[i] = fma2(w.w[3][i], e[u][i],
                    fma2(w.w[2][i], e[u + 1][i], fma2(w.w[1][i], e[u + 2][i], mul2(w.w[0][i], d))));
      }
      const int at = t + u - kHist;
      if (own.value ? u == kHist || t > t0 : at < t1)
        *reinterpret_cast<Raw*>(dxt) = Ch::pack(o);
      else if (own.value && stretch == 0 && dwindow)  // the window's own tokens
        *reinterpret_cast<Raw*>(dwindow + (b * kHist + u) * p.C + c0) = Ch::pack(o);
    }
#pragma unroll
    for (int j = 0; j < kHist; ++j)
#pragma unroll
      for (int i = 0; i < P; ++i) x[j][i] = x[U + j][i], e[j][i] = e[U + j][i];
  };
#pragma unroll
  for (int s = 0; s < kAhead; ++s) fetch(t0 + s * U);
  int t = t0;
  for (; t < t1; t += U) group(t, Flag<true>{});
  group(t, Flag<false>{});
  if constexpr (VEC == 4) asm volatile("cp.async.wait_all;" ::: "memory");
  float* row = part + ((b * stretches + stretch) * p.C + c0) * (kTaps + 1);
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
#pragma unroll
    for (int j = 0; j < kTaps; ++j) row[i * (kTaps + 1) + j] = i & 1 ? dw[j][i / 2].y : dw[j][i / 2].x;
    row[i * (kTaps + 1) + kTaps] = i & 1 ? db[i / 2].y : db[i / 2].x;
  }
}

// Column sums of `count` rows of `width` floats, in a fixed order: 32 columns by 32 row slices
// per block, the slices added at the end.
constexpr int kSumSlices = 32;
template <typename Put>
__device__ __forceinline__ void column_sums(const float* src, int count, int width, int pitch,
                                            Put put) {
  __shared__ float part[kSumSlices][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (c < width)
    for (int r = threadIdx.y; r < count; r += kSumSlices) s += src[(size_t)r * pitch + c];
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < width) {
    float t = 0.f;
    for (int j = 0; j < kSumSlices; ++j) t += part[j][threadIdx.x];
    put(c, t);
  }
}

__global__ void __launch_bounds__(32 * kSumSlices)
    conv_sum_kernel(const float* __restrict__ part, float* __restrict__ dw,
                    float* __restrict__ dbias, int count, int C) {
  column_sums(part, count, C * (kTaps + 1), C * (kTaps + 1), [&](int c, float s) {
    const int ch = c / (kTaps + 1), j = c % (kTaps + 1);
    if (j < kTaps)
      dw[(size_t)ch * kTaps + j] = s;
    else if (dbias)
      dbias[ch] = s;
  });
}

__global__ void __launch_bounds__(32 * kSumSlices)
    sum_rows_kernel(const float* __restrict__ src, float* __restrict__ dst0,
                    float* __restrict__ dst1, int count, int split, int width, int pitch) {
  column_sums(src, count, width, pitch, [&](int c, float s) {
    if (c < split)
      dst0[c] = s;
    else
      dst1[c - split] = s;
  });
}

// Tokens per thread, `span` at most: long stretches re-read little (three tokens each) and sum more in
// registers, short ones give a short prompt enough threads.
int conv_span(int B, int T, int C, int vec, int span) {
  while (span > 8 && (long long)B * ((T + span - 1) / span) * (C / vec) < 152LL * 1024) span /= 2;
  return span;
}

bool rows_aligned(const ConvProblem& p, int vec) {
  const uintptr_t bytes = 2 * vec;
  return p.C % vec == 0 && p.sx.batch % vec == 0 && p.sx.token % vec == 0 &&
         aligned_to(p.x, bytes) && aligned_to(p.window_in, bytes);
}

// Stretches of the backward; a fixed rule of the sizes, so that the workspace can be sized.
int backward_span(int B, int T, int C) { return conv_span(B, T, C, 4, 128); }

template <int VEC>
cudaError_t run_forward(const ConvProblem& p, uint16_t* out, uint16_t* window_out,
                        cudaStream_t stream) {
  const int span = conv_span(p.B, p.T, p.C, VEC, 64);
  const int groups = p.C / VEC, stretches = p.T > 0 ? (p.T + span - 1) / span : 1;
  const long long threads = (long long)groups * stretches * p.B;
  conv_window_kernel<VEC><<<(unsigned)((threads + kThreads - 1) / kThreads), kThreads, 0, stream>>>(
      p, out, window_out, span, groups, stretches);
  return cudaGetLastError();
}

template <int VEC>
cudaError_t run_backward(const ConvProblem& p, const uint16_t* dout, uint16_t* dx,
                         uint16_t* dwindow, float* part, cudaStream_t stream) {
  const int span = backward_span(p.B, p.T, p.C);
  const int groups = p.C / VEC, stretches = (p.T + span - 1) / span;
  const long long threads = (long long)groups * stretches * p.B;
  conv_backward_kernel<VEC>
      <<<(unsigned)((threads + kThreads - 1) / kThreads), kThreads, 0, stream>>>(
          p, dout, dx, dwindow, part, span, groups, stretches);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_sum_rows(const float* src, float* dst0, float* dst1, int count, int split,
                            int width, int pitch, cudaStream_t stream) {
  sum_rows_kernel<<<(width + 31) / 32, dim3(32, kSumSlices), 0, stream>>>(src, dst0, dst1, count,
                                                                          split, width, pitch);
  return cudaGetLastError();
}

cudaError_t launch_conv_window(const ConvProblem& p, uint16_t* out, uint16_t* window_out,
                               cudaStream_t stream) {
  if (rows_aligned(p, 4) && aligned_to(out, 8) && aligned_to(window_out, 8))
    return run_forward<4>(p, out, window_out, stream);
  return run_forward<1>(p, out, window_out, stream);
}

long long conv_backward_rows(int B, int T, int C) {
  const int span = backward_span(B, T, C);
  return (long long)B * ((T + span - 1) / span);
}
size_t conv_backward_workspace_floats(int B, int T, int C) {
  return (size_t)conv_backward_rows(B, T, C) * C * (kTaps + 1);
}

cudaError_t launch_conv_backward(const ConvProblem& p, const uint16_t* dout, uint16_t* dx,
                                 float* dw, float* dbias, uint16_t* dwindow, float* ws,
                                 cudaStream_t stream) {
  cudaError_t err = cudaSuccess;
  int count = 0;
  if (p.T == 0) {
    if (dwindow) err = cudaMemsetAsync(dwindow, 0, (size_t)2 * p.B * kHist * p.C, stream);
  } else {
    const bool vec = rows_aligned(p, 4) && aligned_to(dout, 8) && aligned_to(dx, 8) &&
                     aligned_to(dwindow, 8);
    count = (int)conv_backward_rows(p.B, p.T, p.C);
    err = vec ? run_backward<4>(p, dout, dx, dwindow, ws, stream)
              : run_backward<1>(p, dout, dx, dwindow, ws, stream);
  }
  if (err != cudaSuccess) return err;
  conv_sum_kernel<<<(p.C * (kTaps + 1) + 31) / 32, dim3(32, kSumSlices), 0, stream>>>(
      ws, dw, dbias, count, p.C);
  return cudaGetLastError();
}

}  // namespace m2rnn
