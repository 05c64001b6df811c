// m2rnn_ssm_api.cu — C entries of the selective state space block: argument checks, then the
// launchers.  A failed check launches nothing; nothing here allocates or waits.
#include "../../include/m2rnn.h"
#include "m2rnn_ssm.h"

using namespace m2rnn;

namespace {

m2rnn_status done(cudaError_t e) { return e == cudaSuccess ? M2RNN_OK : M2RNN_ERR_CUDA; }

// Sizes of the scan; the empty sequence is allowed.
m2rnn_status ssm_sizes(int B, int T, int N, int Nqk, int K, int V) {
  if (B < 1 || T < 0 || N < 1 || Nqk < 1 || K < 1 || V < 1 || N % Nqk != 0)
    return M2RNN_ERR_INVALID_ARG;
  if (K > 128 || V > 128 || T > kMaxTokens || (long long)B * N > 0x7fffffffLL) return M2RNN_ERR_UNSUPPORTED;
  return M2RNN_OK;
}
// The backward's too: its sums over parameters count N (2 + V) of them in 32 bits, 32 per block.
m2rnn_status ssm_backward_sizes(int B, int T, int N, int Nqk, int K, int V) {
  const m2rnn_status st = ssm_sizes(B, T, N, Nqk, K, V);
  return st == M2RNN_OK && (long long)N * (2 + V) > 0x7fffffffLL - 31 ? M2RNN_ERR_UNSUPPORTED : st;
}

// Sizes of the convolution; its backward counts 5 C sums, 32 per block, and their rows in 32 bits.
m2rnn_status conv_sizes(int B, int T, int C, bool backward) {
  if (B < 1 || T < 0 || C < 1) return M2RNN_ERR_INVALID_ARG;
  if (T > kMaxTokens || (long long)B * C > 0x7fffffffLL) return M2RNN_ERR_UNSUPPORTED;
  if (backward && (5LL * C > 0x7fffffffLL - 31 || conv_backward_rows(B, T, C) > 0x7fffffffLL))
    return M2RNN_ERR_UNSUPPORTED;
  return M2RNN_OK;
}

// Sizes of the norm; its backward counts 2 D sums, 32 per block, in 32 bits.
m2rnn_status norm_sizes(long long rows, int D, int groups, bool backward) {
  if (rows < 0 || D < 1 || groups < 1 || D % groups != 0) return M2RNN_ERR_INVALID_ARG;
  if (D / groups > kNormMaxGroup || (backward && 2LL * D > 0x7fffffffLL - 31)) return M2RNN_ERR_UNSUPPORTED;
  return M2RNN_OK;
}

// Given strides, or the dense ones.  The stride of a dimension of one is never used: it becomes
// an aligned one.
bool read_strides(const long long* s, int B, int T, int N, int Nqk, int K, int V, Strides (&out)[4]) {
  const long long width[4] = {(long long)Nqk * K, (long long)Nqk * K, (long long)N * V, N};
  for (int i = 0; i < 4; ++i) {
    out[i] = s ? Strides{s[2 * i], s[2 * i + 1]} : Strides{T * width[i], width[i]};
    if (out[i].batch < 0 || out[i].token < 0) return false;
    if (T <= 1) out[i].token = (width[i] + 7) / 8 * 8;
    if (B <= 1) out[i].batch = out[i].token * T;
  }
  return true;
}

}  // namespace

extern "C" {

m2rnn_status m2rnn_conv_silu_window_bf16(const uint16_t* x, const float* w, const float* bias,
                                         const uint16_t* window_in, uint16_t* out,
                                         uint16_t* window_out, int B, int T, int C,
                                         long long x_batch, long long x_token, void* stream) {
  const m2rnn_status st = conv_sizes(B, T, C, false);
  if (st != M2RNN_OK) return st;
  if (!w || x_batch < 0 || x_token < 0) return M2RNN_ERR_INVALID_ARG;
  if (T > 0 && (!x || !out)) return M2RNN_ERR_INVALID_ARG;
  if (!aligned_to(w, 16)) return M2RNN_ERR_INVALID_ARG;
  const ConvProblem p{x, w, bias, window_in, B, T, C, {x_batch, x_token}};
  return done(launch_conv_window(p, out, window_out, static_cast<cudaStream_t>(stream)));
}

size_t m2rnn_conv_silu_backward_workspace_bytes(int B, int T, int C) {
  if (conv_sizes(B, T, C, true) != M2RNN_OK) return 0;
  return sizeof(float) * conv_backward_workspace_floats(B, T, C);
}

m2rnn_status m2rnn_conv_silu_backward_bf16(const uint16_t* x, const float* w, const float* bias,
                                           const uint16_t* window_in, const uint16_t* dout,
                                           uint16_t* dx, float* dw, float* dbias,
                                           uint16_t* dwindow, int B, int T, int C,
                                           long long x_batch, long long x_token, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  const m2rnn_status st = conv_sizes(B, T, C, true);
  if (st != M2RNN_OK) return st;
  if (!w || !dw || x_batch < 0 || x_token < 0) return M2RNN_ERR_INVALID_ARG;
  if (T > 0 && (!x || !dout || !dx || !workspace)) return M2RNN_ERR_INVALID_ARG;
  if (!aligned_to(w, 16) || !aligned_to(workspace, 16)) return M2RNN_ERR_INVALID_ARG;
  if (workspace_bytes < m2rnn_conv_silu_backward_workspace_bytes(B, T, C))
    return M2RNN_ERR_INVALID_ARG;
  const ConvProblem p{x, w, bias, window_in, B, T, C, {x_batch, x_token}};
  return done(launch_conv_backward(p, dout, dx, dw, dbias, dwindow, static_cast<float*>(workspace),
                                   static_cast<cudaStream_t>(stream)));
}

size_t m2rnn_ssm_states_bytes(int B, int T, int N, int K, int V) {
  if (ssm_sizes(B, T, N, 1, K, V) != M2RNN_OK) return 0;
  return (size_t)4 * B * N * (ssm_chunks(T) + 1) * K * V;
}

size_t m2rnn_ssm_workspace_bytes(int B, int T, int N, int Nqk, int K, int V, int backward) {
  if ((backward ? ssm_backward_sizes(B, T, N, Nqk, K, V) : ssm_sizes(B, T, N, Nqk, K, V)) != M2RNN_OK) return 0;
  return backward ? ssm_backward_workspace_bytes(B, T, N, Nqk, K, V)
                  : ssm_forward_workspace_bytes(B, T, N, Nqk, K, V);
}

m2rnn_status m2rnn_ssm_forward_bf16(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                    const uint16_t* a, const float* alpha, const float* beta,
                                    const float* w_r, const float* H0, uint16_t* y, float* H_T,
                                    void* Hs, const long long* strides, int B, int T, int N,
                                    int Nqk, int K, int V, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  const m2rnn_status st = ssm_sizes(B, T, N, Nqk, K, V);
  if (st != M2RNN_OK) return st;
  if (!alpha || !beta || !w_r) return M2RNN_ERR_INVALID_ARG;
  if (T > 0 && (!q || !k || !v || !a || !y)) return M2RNN_ERR_INVALID_ARG;
  Strides s[4];
  if (!read_strides(strides, B, T, N, Nqk, K, V, s)) return M2RNN_ERR_INVALID_ARG;
  const size_t need = ssm_forward_workspace_bytes(B, T, N, Nqk, K, V);
  if (need > 0 && (!workspace || workspace_bytes < need)) return M2RNN_ERR_INVALID_ARG;
  if (!aligned_to(workspace, 16) || !aligned_to(Hs, 16) || !aligned_to(H0, 4) ||
      !aligned_to(H_T, 4))
    return M2RNN_ERR_INVALID_ARG;
  int* status = device_status();
  if (!status) return M2RNN_ERR_CUDA;
  const SsmProblem p{q,    k,    v,    a,    alpha, beta, w_r, H0,  y, H_T, static_cast<uint16_t*>(Hs),
                     s[0], s[1], s[2], s[3], B,     T,    N,   Nqk, K, V,   static_cast<float*>(workspace), status};
  return done(launch_ssm_forward(p, static_cast<cudaStream_t>(stream)));
}

m2rnn_status m2rnn_ssm_backward_bf16(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                     const uint16_t* a, const float* alpha, const float* beta,
                                     const float* w_r, const void* Hs, const uint16_t* dy,
                                     const float* dH_T, uint16_t* dq, uint16_t* dk, uint16_t* dv,
                                     uint16_t* da, float* dalpha, float* dbeta, float* dw_r,
                                     float* dH0, const long long* strides, int B, int T, int N,
                                     int Nqk, int K, int V, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  const m2rnn_status st = ssm_backward_sizes(B, T, N, Nqk, K, V);
  if (st != M2RNN_OK) return st;
  if (!alpha || !beta || !w_r || !dalpha || !dbeta || !dw_r) return M2RNN_ERR_INVALID_ARG;
  if (T > 0 && (!q || !k || !v || !a || !Hs || !dy || !dq || !dk || !dv || !da))
    return M2RNN_ERR_INVALID_ARG;
  Strides s[4];
  if (!read_strides(strides, B, T, N, Nqk, K, V, s)) return M2RNN_ERR_INVALID_ARG;
  const size_t need = ssm_backward_workspace_bytes(B, T, N, Nqk, K, V);
  if (need > 0 && (!workspace || workspace_bytes < need)) return M2RNN_ERR_INVALID_ARG;
  if (!aligned_to(workspace, 16) || !aligned_to(Hs, 16) || !aligned_to(dH_T, 4) ||
      !aligned_to(dH0, 4))
    return M2RNN_ERR_INVALID_ARG;
  int* status = device_status();
  if (!status) return M2RNN_ERR_CUDA;
  const SsmBackwardProblem p{q,  k,  v,  a,  alpha,  beta,  w_r,  static_cast<const uint16_t*>(Hs),
                             dy, dH_T, dq, dk, dv, da, dalpha, dbeta, dw_r, dH0, s[0], s[1], s[2],
                             s[3], B, T, N, Nqk, K, V, static_cast<float*>(workspace), status};
  return done(launch_ssm_backward(p, static_cast<cudaStream_t>(stream)));
}

m2rnn_status m2rnn_ssm_step_bf16(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                 const uint16_t* a, const float* alpha, const float* beta,
                                 const float* w_r, const float* H_in, float* H_out, uint16_t* y,
                                 int B, int N, int Nqk, int K, int V, void* stream) {
  const m2rnn_status st = ssm_sizes(B, 1, N, Nqk, K, V);
  if (st != M2RNN_OK) return st;
  if (!q || !k || !v || !a || !alpha || !beta || !w_r || !H_out || !y)
    return M2RNN_ERR_INVALID_ARG;
  return done(launch_ssm_step(q, k, v, a, alpha, beta, w_r, H_in, H_out, y, B, N, Nqk, K, V,
                              static_cast<cudaStream_t>(stream)));
}

m2rnn_status m2rnn_gate_groupnorm(const void* y, int y_f32, const uint16_t* g_pre, const float* w,
                                  const float* bias, float eps, uint16_t* out, long long rows,
                                  int D, int groups, void* stream) {
  const m2rnn_status st = norm_sizes(rows, D, groups, false);
  if (st != M2RNN_OK) return st;
  if (!(eps >= 0.f) || !w) return M2RNN_ERR_INVALID_ARG;
  if (rows == 0) return M2RNN_OK;
  if (!y || !out) return M2RNN_ERR_INVALID_ARG;
  const NormProblem p{y, y_f32 != 0, g_pre, w, bias, eps, rows, D, groups};
  return done(launch_groupnorm(p, out, static_cast<cudaStream_t>(stream)));
}

size_t m2rnn_gate_groupnorm_backward_workspace_bytes(long long rows, int D, int groups) {
  if (norm_sizes(rows, D, groups, true) != M2RNN_OK) return 0;
  return sizeof(float) * groupnorm_backward_workspace_floats(rows, D, groups);
}

m2rnn_status m2rnn_gate_groupnorm_backward(const void* y, int y_f32, const uint16_t* g_pre,
                                           const float* w, const float* bias, float eps,
                                           const uint16_t* dout, void* dy, uint16_t* dg_pre,
                                           float* dw, float* dbias, long long rows, int D,
                                           int groups, void* workspace, size_t workspace_bytes,
                                           void* stream) {
  const m2rnn_status st = norm_sizes(rows, D, groups, true);
  if (st != M2RNN_OK) return st;
  if (!(eps >= 0.f) || !w || !dw) return M2RNN_ERR_INVALID_ARG;
  if (rows > 0 && (!y || !dout || !dy || !workspace || (g_pre != nullptr) != (dg_pre != nullptr)))
    return M2RNN_ERR_INVALID_ARG;
  if (!aligned_to(workspace, 16) ||
      workspace_bytes < m2rnn_gate_groupnorm_backward_workspace_bytes(rows, D, groups))
    return M2RNN_ERR_INVALID_ARG;
  const NormProblem p{y, y_f32 != 0, g_pre, w, bias, eps, rows, D, groups};
  return done(launch_groupnorm_backward(p, dout, dy, dg_pre, dw, dbias,
                                        static_cast<float*>(workspace),
                                        static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
