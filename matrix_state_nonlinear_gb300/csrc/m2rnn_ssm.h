// m2rnn_ssm.h — the selective state space block's kernels: problem descriptions shared by
// the C entries (m2rnn_ssm_api.cu) and the launchers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace m2rnn {

constexpr int kSsmChunk = 128;   // tokens per chunk of the scan
constexpr int kSsmColumns = 64;  // value columns per block of the scan

// Tokens of a sequence at most: counts of them are rounded up to stretches of 128 in 32 bits.
constexpr int kMaxTokens = 0x7fffffff - 127;

// Batch and token strides of one bf16 operand, in elements.
struct Strides {
  long long batch, token;
};

// Device address of the current device's status word (m2rnn_stream_status), or null.
int* device_status();

struct SsmProblem {
  const uint16_t *q, *k, *v, *a;
  const float *alpha, *beta, *w_r, *H0;
  uint16_t* y;
  float* H_T;
  uint16_t* Hs;  // [B, N, chunks + 1, 2 (high, low), K, V], or null
  Strides sq, sk, sv, sa;
  int B, T, N, Nqk, K, V;
  float* ws;
  int* status;
};

struct SsmBackwardProblem {
  const uint16_t *q, *k, *v, *a;
  const float *alpha, *beta, *w_r;
  const uint16_t* Hs;
  const uint16_t* dy;
  const float* dH_T;
  uint16_t *dq, *dk, *dv, *da;
  float *dalpha, *dbeta, *dw_r, *dH0;
  Strides sq, sk, sv, sa;
  int B, T, N, Nqk, K, V;
  float* ws;
  int* status;
};

__host__ __device__ inline int ssm_chunks(int T) { return (T + kSsmChunk - 1) / kSsmChunk; }

// A pair's chunks are cut into `segments` of `per` chunks that run side by side.
struct SsmCut {
  int segments, per;
};
SsmCut ssm_cut(int B, int T, int N, int V);
size_t ssm_segment_floats(const SsmCut& c, int B, int N, int K, int V);

// The state's sums alone (m2rnn_ssm_state.cu).
struct StateProblem {
  const uint16_t *x, *y;  // k and v, or, backwards, q and dy
  const uint16_t* a;
  const float *alpha, *beta;
  Strides sx, sy, sa;
  int B, T, N, Nqk, K, V;
  const float* from;        // the first state (backwards: the last one's gradient), or null
  const float* from_state;  // or every segment's, [pairs][segments][K][V]
  float* to;                // the last state (backwards: the first one's gradient), or null
  uint16_t* kept;           // the state before every chunk and the last, [pairs][chunks + 1][2 (high,
                            // low)][K][V]; backwards: G after every chunk, [pairs][chunks][2][K][V]
  const uint16_t* Hs;       // with that: the forward's states,
  float* dots;              // and <G, H before the chunk>, [pairs][chunks][tiles of V][8 parts]
  int* status;
  int pieces, per, first_piece;  // set by the launches, as are
  float *to_state, *decay;
};
// Every segment's starting state (backwards: its last state's gradient) into ws,
// ssm_segment_floats.
cudaError_t launch_ssm_segments(StateProblem p, const SsmCut& c, bool reverse, bool vec, float* ws,
                                cudaStream_t stream);
// kept (backwards: dots too) and `to`, from `from` or from_state.
cudaError_t launch_ssm_kept_states(StateProblem p, const SsmCut& c, bool reverse, bool vec, cudaStream_t stream);

size_t ssm_forward_workspace_bytes(int B, int T, int N, int Nqk, int K, int V);
size_t ssm_backward_workspace_bytes(int B, int T, int N, int Nqk, int K, int V);
cudaError_t launch_ssm_forward(const SsmProblem& p, cudaStream_t stream);
cudaError_t launch_ssm_backward(const SsmBackwardProblem& p, cudaStream_t stream);
cudaError_t launch_ssm_step(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                            const uint16_t* a, const float* alpha, const float* beta,
                            const float* w_r, const float* H_in, float* H_out, uint16_t* y, int B,
                            int N, int Nqk, int K, int V, cudaStream_t stream);

struct ConvProblem {
  const uint16_t* x;
  const float *w, *bias;
  const uint16_t* window_in;
  int B, T, C;
  Strides sx;
};
cudaError_t launch_conv_window(const ConvProblem& p, uint16_t* out, uint16_t* window_out,
                               cudaStream_t stream);
size_t conv_backward_workspace_floats(int B, int T, int C);
long long conv_backward_rows(int B, int T, int C);  // of partial sums, 5 C floats each
cudaError_t launch_conv_backward(const ConvProblem& p, const uint16_t* dout, uint16_t* dx,
                                 float* dw, float* dbias, uint16_t* dwindow, float* ws,
                                 cudaStream_t stream);

struct NormProblem {
  const void* y;
  bool y_f32;
  const uint16_t* g;
  const float *w, *bias;
  float eps;
  long long rows;
  int D, groups;
};
constexpr int kNormMaxGroup = 8192;  // channels per group
cudaError_t launch_groupnorm(const NormProblem& p, uint16_t* out, cudaStream_t stream);
size_t groupnorm_backward_workspace_floats(long long rows, int D, int groups);
cudaError_t launch_groupnorm_backward(const NormProblem& p, const uint16_t* dout, void* dy,
                                      uint16_t* dg, float* dw, float* dbias, float* ws,
                                      cudaStream_t stream);

// Sums the first `width` columns of `count` rows (row r at src + r * pitch) in a fixed order:
// column c goes to dst0[c] for c < split, to dst1[c - split] after that.
cudaError_t launch_sum_rows(const float* src, float* dst0, float* dst1, int count, int split,
                            int width, int pitch, cudaStream_t stream);

inline bool aligned_to(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) % n) == 0;
}
// Rows of `width` bf16 values that can be read 16 bytes at a time.
inline bool rows_of_16(const void* p, const Strides& s, int width) {
  return width % 8 == 0 && s.batch % 8 == 0 && s.token % 8 == 0 && aligned_to(p, 16);
}

#ifdef __CUDACC__
// The gate of one token: d = softplus(x), log f = -alpha d, x = a + beta.  log f is held at
// -105 and above: exp(-105) is zero in float32 already, and the sums over a chunk of 128 tokens
// are bounded (ChunkGates).
__device__ __forceinline__ float2 ssm_gate(float a, float alpha, float beta) {
  const float x = a + beta;
  const float d = fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
  return make_float2(d, fmaxf(-alpha * d, -105.f));
}
// sigmoid(x) / softplus(x), the limit 1 included (x -> -infinity).
__device__ __forceinline__ float sigmoid_over_softplus(float x) {
  const float e = expf(-fabsf(x));
  const float sig = x >= 0.f ? 1.f / (1.f + e) : e / (1.f + e);
  return x < -17.f ? 1.f : sig / (fmaxf(x, 0.f) + log1pf(e));
}
__device__ __forceinline__ float bf16_to_f(uint16_t u) {
  return __uint_as_float(static_cast<uint32_t>(u) << 16);
}
__device__ __forceinline__ uint16_t f_to_bf16(float f) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(f));
}
#endif

}  // namespace m2rnn
