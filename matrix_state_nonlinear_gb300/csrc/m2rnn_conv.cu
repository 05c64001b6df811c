// m2rnn_conv.cu — the short causal convolution (4 taps, depthwise, SiLU) with a carried window,
// and its backward pass.
//
//   pre[t] = bias + sum_j w[j] X[t-3+j],  out = pre sigmoid(pre),  X = window then x
//   dpre[t] = dout[t] sigma (1 + pre (1 - sigma))
//   dX[t] = sum_j w[j] dpre[t+3-j],  dw[j] = sum_{b,t} dpre[t] X[t-3+j],  dbias = sum dpre
//
// Memory-bound: the forward reads and writes every element once (4 bytes an element), the
// backward reads two and writes one (6 bytes).  A thread owns kVec neighbouring channels over a
// stretch of tokens and slides a window of three tokens through registers; eight tokens are
// loaded ahead of their arithmetic so that enough bytes are in flight.
#include "m2rnn_ssm.h"
#include "ptx_util.cuh"

namespace m2rnn {
namespace {

constexpr int kTaps = 4;
constexpr int kHist = kTaps - 1;
constexpr int kThreads = 128;

template <int VEC>
struct Raw;  // VEC bf16 values as loaded
template <>
struct Raw<8> {
  uint4 u;
};
template <>
struct Raw<4> {
  uint2 u;
};
template <>
struct Raw<1> {
  uint16_t u;
};

template <int VEC>
__device__ __forceinline__ Raw<VEC> load_raw(const uint16_t* p) {
  return *reinterpret_cast<const Raw<VEC>*>(p);
}
__device__ __forceinline__ void unpack(const Raw<8>& r, float (&f)[8]) {
  f[0] = bf16_lo(r.u.x), f[1] = bf16_hi(r.u.x), f[2] = bf16_lo(r.u.y), f[3] = bf16_hi(r.u.y);
  f[4] = bf16_lo(r.u.z), f[5] = bf16_hi(r.u.z), f[6] = bf16_lo(r.u.w), f[7] = bf16_hi(r.u.w);
}
__device__ __forceinline__ void unpack(const Raw<4>& r, float (&f)[4]) {
  f[0] = bf16_lo(r.u.x), f[1] = bf16_hi(r.u.x), f[2] = bf16_lo(r.u.y), f[3] = bf16_hi(r.u.y);
}
__device__ __forceinline__ void unpack(const Raw<1>& r, float (&f)[1]) { f[0] = bf16_to_f(r.u); }
__device__ __forceinline__ void store_vec(uint16_t* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                            pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void store_vec(uint16_t* p, const float (&f)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}
__device__ __forceinline__ void store_vec(uint16_t* p, const float (&f)[1]) { *p = f_to_bf16(f[0]); }

// sigmoid with the fast exponential: relative error a few 2^-22, below the bf16 rounding of
// every result but the sums dw and dbias, where it stays below 1e-6 of them.
__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// X[t] of one batch row: the window for t in [-3, -1], x after that.
template <int VEC>
__device__ __forceinline__ void load_x(const uint16_t* xb, const uint16_t* win, long long x_token,
                                       int C, int t, float (&f)[VEC]) {
  if (t >= 0) {
    unpack(load_raw<VEC>(xb + t * x_token), f);
  } else if (win) {
    unpack(load_raw<VEC>(win + (long long)(t + kHist) * C), f);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = 0.f;
  }
}

template <int VEC>
__device__ __forceinline__ void load_taps(const float* w, const float* bias, int c0,
                                          float (&wt)[VEC][kTaps], float (&bs)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const float4 u = *reinterpret_cast<const float4*>(w + (size_t)(c0 + i) * kTaps);
    wt[i][0] = u.x, wt[i][1] = u.y, wt[i][2] = u.z, wt[i][3] = u.w;
    bs[i] = bias ? bias[c0 + i] : 0.f;
  }
}

// Forward: one thread, VEC channels, `span` tokens of one batch row.  The thread of the first
// stretch also writes the window after x: it alone reads window_in, so that the two may be the
// same memory.
template <int VEC>
__global__ void __launch_bounds__(kThreads)
    conv_window_kernel(ConvProblem p, uint16_t* __restrict__ out, uint16_t* window_out, int span,
                       int groups, int stretches) {
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int c0 = VEC * (int)(id % groups);
  const int stretch = (int)(id / groups % stretches);
  const long long b = id / groups / stretches;
  if (b >= p.B) return;
  float wt[VEC][kTaps], bs[VEC];
  load_taps<VEC>(p.w, p.bias, c0, wt, bs);
  const uint16_t* xb = p.x + b * p.sx.batch + c0;
  const uint16_t* win = p.window_in ? p.window_in + b * kHist * p.C + c0 : nullptr;
  uint16_t* ob = out + b * p.T * p.C + c0;
  const int t0 = stretch * span, t1 = min(p.T, t0 + span);
  float h[kHist][VEC];  // X[t-3], X[t-2], X[t-1]
#pragma unroll
  for (int j = 0; j < kHist; ++j) load_x<VEC>(xb, win, p.sx.token, p.C, t0 - kHist + j, h[j]);
  if (stretch == 0 && window_out) {
    float f[kHist][VEC];
#pragma unroll
    for (int j = 0; j < kHist; ++j) load_x<VEC>(xb, win, p.sx.token, p.C, p.T - kHist + j, f[j]);
#pragma unroll
    for (int j = 0; j < kHist; ++j) store_vec(window_out + (b * kHist + j) * p.C + c0, f[j]);
  }
  constexpr int kAhead = 8;
  for (int t = t0; t < t1; t += kAhead) {
    Raw<VEC> raw[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (t + u < t1) raw[u] = load_raw<VEC>(xb + (t + u) * p.sx.token);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (t + u >= t1) break;
      float x[VEC], o[VEC];
      unpack(raw[u], x);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        float s = bs[i];
        s = fmaf(wt[i][0], h[0][i], s);
        s = fmaf(wt[i][1], h[1][i], s);
        s = fmaf(wt[i][2], h[2][i], s);
        s = fmaf(wt[i][3], x[i], s);
        o[i] = s * sigmoid_f(s);
        h[0][i] = h[1][i], h[1][i] = h[2][i], h[2][i] = x[i];
      }
      store_vec(ob + (long long)(t + u) * p.C, o);
    }
  }
}

// Backward: one thread, VEC channels, `span` tokens of one batch row.  dX[t] needs dpre up to
// t + 3, so the thread runs three tokens past its stretch; only its own tokens enter dw, dbias.
// The partial sums of each (batch row, stretch) go to `part` [rows][C][5].
template <int VEC>
__global__ void __launch_bounds__(kThreads)
    conv_backward_kernel(ConvProblem p, const uint16_t* __restrict__ dout,
                         uint16_t* __restrict__ dx, uint16_t* __restrict__ dwindow,
                         float* __restrict__ part, int span, int groups, int stretches) {
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int c0 = VEC * (int)(id % groups);
  const int stretch = (int)(id / groups % stretches);
  const long long b = id / groups / stretches;
  if (b >= p.B) return;
  float wt[VEC][kTaps], bs[VEC];
  load_taps<VEC>(p.w, p.bias, c0, wt, bs);
  const uint16_t* xb = p.x + b * p.sx.batch + c0;
  const uint16_t* win = p.window_in ? p.window_in + b * kHist * p.C + c0 : nullptr;
  const uint16_t* gb = dout + b * p.T * p.C + c0;
  uint16_t* dxb = dx + b * p.T * p.C + c0;
  const int t0 = stretch * span, t1 = min(p.T, t0 + span);
  float h[kHist][VEC], e[kHist][VEC];  // X[t-3..t-1], dpre[t-3..t-1] (zero before the stretch)
  float dw[VEC][kTaps], db[VEC];
#pragma unroll
  for (int j = 0; j < kHist; ++j) {
    load_x<VEC>(xb, win, p.sx.token, p.C, t0 - kHist + j, h[j]);
#pragma unroll
    for (int i = 0; i < VEC; ++i) e[j][i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    db[i] = 0.f;
#pragma unroll
    for (int j = 0; j < kTaps; ++j) dw[i][j] = 0.f;
  }
  // At token t, dX[t-3] is complete: from dpre[t-3..t].  It is this thread's for t - 3 >= t0, or
  // the window's for t - 3 < 0.
  constexpr int kAhead = 4;
  const int tend = t1 + kHist;
  for (int t = t0; t < tend; t += kAhead) {
    Raw<VEC> xr[kAhead], gr[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (t + u < tend && t + u < p.T) {
        xr[u] = load_raw<VEC>(xb + (t + u) * p.sx.token);
        gr[u] = load_raw<VEC>(gb + (long long)(t + u) * p.C);
      }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int tt = t + u;
      if (tt >= tend) break;
      float x[VEC], g[VEC], o[VEC];
      if (tt < p.T) {
        unpack(xr[u], x);
        unpack(gr[u], g);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = g[i] = 0.f;
      }
      const bool mine = tt < t1;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        float s = bs[i];
        s = fmaf(wt[i][0], h[0][i], s);
        s = fmaf(wt[i][1], h[1][i], s);
        s = fmaf(wt[i][2], h[2][i], s);
        s = fmaf(wt[i][3], x[i], s);
        const float sig = sigmoid_f(s);
        const float d = tt < p.T ? g[i] * (sig * fmaf(s, 1.f - sig, 1.f)) : 0.f;
        if (mine) {
          db[i] += d;
          dw[i][0] = fmaf(d, h[0][i], dw[i][0]);
          dw[i][1] = fmaf(d, h[1][i], dw[i][1]);
          dw[i][2] = fmaf(d, h[2][i], dw[i][2]);
          dw[i][3] = fmaf(d, x[i], dw[i][3]);
        }
        o[i] = fmaf(wt[i][3], e[0][i],
                    fmaf(wt[i][2], e[1][i], fmaf(wt[i][1], e[2][i], wt[i][0] * d)));
        h[0][i] = h[1][i], h[1][i] = h[2][i], h[2][i] = x[i];
        e[0][i] = e[1][i], e[1][i] = e[2][i], e[2][i] = d;
      }
      if (tt - kHist >= t0)
        store_vec(dxb + (long long)(tt - kHist) * p.C, o);
      else if (stretch == 0 && dwindow)  // tt < 3 in the first stretch: the window's own tokens
        store_vec(dwindow + (b * kHist + tt) * p.C + c0, o);
    }
  }
  if (part) {
    float* row = part + ((b * stretches + stretch) * p.C + c0) * (kTaps + 1);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
      for (int j = 0; j < kTaps; ++j) row[i * (kTaps + 1) + j] = dw[i][j];
      row[i * (kTaps + 1) + kTaps] = db[i];
    }
  }
}

// Column sums of `count` rows of `width` floats, in a fixed order: 32 columns by 8 row slices
// per block, the slices added at the end.
constexpr int kSumSlices = 8;
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
#pragma unroll
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

// Tokens per thread: long stretches re-read little (three tokens each) and sum more in
// registers, short ones give a short prompt enough threads.
int conv_span(int B, int T, int C, int vec) {
  int span = 64;
  while (span > 8 && (long long)B * ((T + span - 1) / span) * (C / vec) < 152LL * 1024) span /= 2;
  return span;
}

bool rows_aligned(const ConvProblem& p, int vec) {
  const uintptr_t bytes = 2 * vec;
  return p.C % vec == 0 && p.sx.batch % vec == 0 && p.sx.token % vec == 0 &&
         aligned_to(p.x, bytes) && aligned_to(p.window_in, bytes);
}

// Stretches of the backward; a fixed rule of the sizes, so that the workspace can be sized.
int backward_span(int B, int T, int C) { return conv_span(B, T, C, 4); }

template <int VEC>
cudaError_t run_forward(const ConvProblem& p, uint16_t* out, uint16_t* window_out,
                        cudaStream_t stream) {
  const int span = conv_span(p.B, p.T, p.C, VEC);
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
  if (rows_aligned(p, 8) && aligned_to(out, 16) && aligned_to(window_out, 16))
    return run_forward<8>(p, out, window_out, stream);
  return run_forward<1>(p, out, window_out, stream);
}

size_t conv_backward_workspace_floats(int B, int T, int C) {
  const int span = backward_span(B, T, C);
  return (size_t)B * ((T + span - 1) / span) * C * (kTaps + 1);
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
    const int span = backward_span(p.B, p.T, p.C);
    count = p.B * ((p.T + span - 1) / span);
    err = vec ? run_backward<4>(p, dout, dx, dwindow, ws, stream)
              : run_backward<1>(p, dout, dx, dwindow, ws, stream);
  }
  if (err != cudaSuccess) return err;
  conv_sum_kernel<<<(p.C * (kTaps + 1) + 31) / 32, dim3(32, kSumSlices), 0, stream>>>(
      ws, dw, dbias, count, p.C);
  return cudaGetLastError();
}

}  // namespace m2rnn
