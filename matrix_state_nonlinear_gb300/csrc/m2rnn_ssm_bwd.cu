// m2rnn_ssm_bwd.cu — gradients of the selective scan, token by token (see include/m2rnn.h).
//
// One block per (batch, head) pair walks the chunks in reverse: it recomputes the chunk's states
// from the kept one into the workspace, then scans its tokens in reverse with the state's
// gradient in shared memory.  Per-head dq, dk and per-pair parameter sums go to the workspace
// and are added in a fixed order.
#include "m2rnn_ssm.h"

namespace m2rnn {
namespace {

constexpr int kThreads = 128;

struct Workspace {
  float *hist, *dq, *dk, *par;  // [pairs][65][K][V], [B,T,N,K] x 2, [pairs][2 + V]
  size_t floats;
};
Workspace carve(float* ws, int B, int T, int N, int K, int V) {
  const size_t pairs = (size_t)B * N, kv = (size_t)K * V, tok = (size_t)B * T * N * K;
  Workspace w;
  w.hist = ws;
  w.dq = w.hist + pairs * (kSsmChunk + 1) * kv;
  w.dk = w.dq + tok;
  w.par = w.dk + tok;
  w.floats = pairs * (kSsmChunk + 1) * kv + 2 * tok + pairs * (2 + V);
  return w;
}

__device__ __forceinline__ float block_sum(float s) {
  __shared__ float part[kThreads];
  __syncthreads();
  part[threadIdx.x] = s;
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < kThreads; ++i) t += part[i];
  return t;
}

__global__ void __launch_bounds__(kThreads) ssm_backward_kernel(SsmBackwardProblem p, Workspace w) {
  extern __shared__ float G[];  // [K][V]
  __shared__ float sk[128], sq[128], sv[128], sdy[128];
  const long long pair = blockIdx.x;
  const int n = (int)(pair % p.N), c = threadIdx.x, K = p.K, V = p.V;
  const long long b = pair / p.N;
  const int head = (int)((long long)n * p.Nqk / p.N);
  const int chunks = ssm_chunks(p.T);
  const size_t KV = (size_t)K * V;
  const bool live = c < V, krow = c < K;
  float* hist = w.hist + (size_t)pair * (kSsmChunk + 1) * KV;
  const float alpha = p.alpha[n], beta = p.beta[n];
  const float wr = live ? p.w_r[(size_t)n * V + c] : 0.f;
  for (int i = 0; i < K && live; ++i)
    G[i * V + c] = p.dH_T ? p.dH_T[pair * KV + (size_t)i * V + c] : 0.f;
  auto token = [&](int t, bool dy) {
    __syncthreads();
    if (krow) {
      sk[c] = bf16_to_f(p.k[b * p.sk.batch + t * p.sk.token + (size_t)head * K + c]);
      sq[c] = bf16_to_f(p.q[b * p.sq.batch + t * p.sq.token + (size_t)head * K + c]);
    }
    if (live) {
      sv[c] = bf16_to_f(p.v[b * p.sv.batch + t * p.sv.token + (size_t)n * V + c]);
      if (dy) sdy[c] = bf16_to_f(p.dy[((b * p.T + t) * p.N + n) * V + c]);
    }
    __syncthreads();
  };
  float dalpha = 0.f, dbeta = 0.f, dwr = 0.f;
  for (int chunk = chunks - 1; chunk >= 0; --chunk) {
    const int t0 = chunk * kSsmChunk, t1 = min(p.T, t0 + kSsmChunk);
    const uint16_t* s = p.Hs + ((size_t)pair * (chunks + 1) + chunk) * 2 * KV;
    for (int i = 0; i < K && live; ++i)
      hist[(size_t)i * V + c] =
          bf16_to_f(s[(size_t)i * V + c]) + bf16_to_f(s[KV + (size_t)i * V + c]);
    for (int t = t0; t < t1; ++t) {
      token(t, false);
      const float2 gate = ssm_gate(bf16_to_f(p.a[b * p.sa.batch + t * p.sa.token + n]), alpha, beta);
      const float f = expf(gate.y);
      const float* h = hist + (size_t)(t - t0) * KV;
      for (int i = 0; i < K && live; ++i)
        hist[(size_t)(t - t0 + 1) * KV + (size_t)i * V + c] =
            fmaf(f, h[(size_t)i * V + c], gate.x * sk[i] * sv[c]);
    }
    for (int t = t1 - 1; t >= t0; --t) {
      token(t, true);
      const float x = bf16_to_f(p.a[b * p.sa.batch + t * p.sa.token + n]) + beta;
      const float2 gate = ssm_gate(x - beta, alpha, beta);
      const float d = gate.x, f = expf(gate.y);
      const float* hb = hist + (size_t)(t - t0) * KV;
      const float* ha = hb + KV;
      float dv = 0.f, g = 0.f;
      for (int i = 0; i < K && live; ++i) {
        const float gi = fmaf(sq[i], sdy[c], G[i * V + c]);
        G[i * V + c] = gi;
        dv = fmaf(gi, sk[i], dv);
        g = fmaf(gi, hb[(size_t)i * V + c], g);
      }
      g = f * block_sum(g);
      const size_t at = ((size_t)(b * p.T + t) * p.N + n);
      float kgv = 0.f;
      if (krow) {
        float dq = 0.f, gv = 0.f;
        for (int j = 0; j < V; ++j) {
          dq = fmaf(ha[(size_t)c * V + j], sdy[j], dq);
          gv = fmaf(G[c * V + j], sv[j], gv);
        }
        w.dq[at * K + c] = dq;
        w.dk[at * K + c] = d * gv;
        kgv = sk[c] * gv;
      }
      kgv = block_sum(kgv);
      const float sig = 1.f / (1.f + expf(-x));
      const float da = sig * (kgv - alpha * g);
      if (c == 0) p.da[at] = f_to_bf16(da);
      dalpha -= d * g;
      dbeta += da;
      if (live) {
        p.dv[at * V + c] = f_to_bf16(fmaf(wr, sdy[c], d * dv));
        dwr = fmaf(sdy[c], sv[c], dwr);
        for (int i = 0; i < K; ++i) G[i * V + c] *= f;
      }
    }
    __syncthreads();
  }
  float* par = w.par + pair * (2 + V);
  if (c == 0) par[0] = dalpha, par[1] = dbeta;
  if (live) par[2 + c] = dwr;
  for (int i = 0; i < K && live && p.dH0; ++i) p.dH0[pair * KV + (size_t)i * V + c] = G[i * V + c];
}

// dq, dk of one (token, q/k head): the sum over the heads that read it.
__global__ void __launch_bounds__(256)
    sum_heads_kernel(SsmBackwardProblem p, Workspace w) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= (long long)p.B * p.T * p.Nqk * p.K) return;
  const int rep = p.N / p.Nqk, k = (int)(i % p.K);
  const long long at = i / p.K;  // (b, t, head)
  float dq = 0.f, dk = 0.f;
  for (int r = 0; r < rep; ++r) {
    dq += w.dq[(at * rep + r) * p.K + k];
    dk += w.dk[(at * rep + r) * p.K + k];
  }
  p.dq[i] = f_to_bf16(dq);
  p.dk[i] = f_to_bf16(dk);
}

__global__ void __launch_bounds__(128) sum_params_kernel(SsmBackwardProblem p, const float* par) {
  const int n = blockIdx.x;
  for (int c = threadIdx.x; c < 2 + p.V; c += 128) {
    float s = 0.f;
    for (int b = 0; b < p.B && p.T > 0; ++b) s += par[((size_t)b * p.N + n) * (2 + p.V) + c];
    if (c == 0)
      p.dalpha[n] = s;
    else if (c == 1)
      p.dbeta[n] = s;
    else
      p.dw_r[(size_t)n * p.V + c - 2] = s;
  }
}

}  // namespace

size_t ssm_backward_workspace_bytes(int B, int T, int N, int, int K, int V) {
  return sizeof(float) * carve(nullptr, B, T, N, K, V).floats;
}

cudaError_t launch_ssm_backward(const SsmBackwardProblem& p, cudaStream_t stream) {
  const Workspace w = carve(p.ws, p.B, p.T, p.N, p.K, p.V);
  const int smem = (int)sizeof(float) * p.K * p.V;
  cudaError_t err = cudaFuncSetAttribute(ssm_backward_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  ssm_backward_kernel<<<(unsigned)((long long)p.B * p.N), kThreads, smem, stream>>>(p, w);
  const long long n = (long long)p.B * p.T * p.Nqk * p.K;
  if (n > 0)
    sum_heads_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(p, w);
  sum_params_kernel<<<p.N, 128, 0, stream>>>(p, w.par);
  return cudaGetLastError();
}

}  // namespace m2rnn
