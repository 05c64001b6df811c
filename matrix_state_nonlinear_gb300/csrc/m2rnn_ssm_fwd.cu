// m2rnn_ssm_fwd.cu — the selective scan of a prompt, token by token (see include/m2rnn.h).
//
// One block per (batch, head) pair; thread v owns column v of the state, held in shared memory.
#include "m2rnn_ssm.h"

namespace m2rnn {
namespace {

constexpr int kThreads = 128;

__global__ void __launch_bounds__(kThreads) ssm_forward_kernel(SsmProblem p) {
  extern __shared__ float H[];  // [K][V]
  __shared__ float sk[128], sq[128];
  const long long pair = blockIdx.x;
  const int n = (int)(pair % p.N), c = threadIdx.x;
  const long long b = pair / p.N;
  const int head = (int)((long long)n * p.Nqk / p.N);
  const int chunks = ssm_chunks(p.T);
  const size_t KV = (size_t)p.K * p.V;
  const bool live = c < p.V;
  for (int i = 0; i < p.K && live; ++i)
    H[i * p.V + c] = p.H0 ? p.H0[pair * KV + (size_t)i * p.V + c] : 0.f;
  auto keep = [&](int chunk) {
    if (!p.Hs || !live) return;
    uint16_t* s = p.Hs + ((size_t)pair * (chunks + 1) + chunk) * 2 * KV;
    for (int i = 0; i < p.K; ++i) {
      const float h = H[i * p.V + c];
      const uint16_t hi = f_to_bf16(h);
      s[(size_t)i * p.V + c] = hi;
      s[KV + (size_t)i * p.V + c] = f_to_bf16(h - bf16_to_f(hi));
    }
  };
  for (int t = 0; t < p.T; ++t) {
    if (t % kSsmChunk == 0) keep(t / kSsmChunk);
    __syncthreads();
    if (c < p.K) {
      sk[c] = bf16_to_f(p.k[b * p.sk.batch + t * p.sk.token + (size_t)head * p.K + c]);
      sq[c] = bf16_to_f(p.q[b * p.sq.batch + t * p.sq.token + (size_t)head * p.K + c]);
    }
    __syncthreads();
    if (!live) continue;
    const float2 gate =
        ssm_gate(bf16_to_f(p.a[b * p.sa.batch + t * p.sa.token + n]), p.alpha[n], p.beta[n]);
    const float f = expf(gate.y);
    const float v = bf16_to_f(p.v[b * p.sv.batch + t * p.sv.token + (size_t)n * p.V + c]);
    float y = 0.f;
    for (int i = 0; i < p.K; ++i) {
      const float h = fmaf(f, H[i * p.V + c], gate.x * sk[i] * v);
      H[i * p.V + c] = h;
      y = fmaf(h, sq[i], y);
    }
    p.y[((b * p.T + t) * p.N + n) * p.V + c] = f_to_bf16(fmaf(p.w_r[(size_t)n * p.V + c], v, y));
  }
  keep(chunks);
  for (int i = 0; i < p.K && live && p.H_T; ++i)
    p.H_T[pair * KV + (size_t)i * p.V + c] = H[i * p.V + c];
}

}  // namespace

size_t ssm_forward_workspace_bytes(int, int, int, int, int, int) { return 0; }

cudaError_t launch_ssm_forward(const SsmProblem& p, cudaStream_t stream) {
  const int smem = (int)sizeof(float) * p.K * p.V;
  cudaError_t err = cudaFuncSetAttribute(ssm_forward_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  ssm_forward_kernel<<<(unsigned)((long long)p.B * p.N), kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace m2rnn
