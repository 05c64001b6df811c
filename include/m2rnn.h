/*
 * m2rnn.h — C ABI of the GB300 (sm_103a) M²RNN forward-recurrence library.
 *
 * What it computes.  The forward pass of the M²RNN matrix-state nonlinear
 * recurrence, as stated in the M²RNN study notes ("M²RNN: 矩阵状态非线性 RNN
 * 的容量、表达力与系统代价", notes on arXiv:2603.14360v2):
 *   Sec. 2.2, Eq. (13)/(17):  f_t = exp(-alpha_n * softplus(a_t + beta_n))
 *   Sec. 2.1, Eq. (10):       Z_t = tanh(H_{t-1} W_n + k_t v_t^T)
 *             Eq. (11):       H_t = f_t H_{t-1} + (1 - f_t) Z_t
 *             Eq. (12):       y_t = H_t^T q_t + w_r ⊙ v_t
 * for every (batch b, head n) independently (Sec. 2.6: each (b, n) pair is an
 * independent work unit), starting from H_0 (zero when not given).
 *
 * Layout.  Every tensor is dense and row-major (innermost index last):
 *   q, k   [B, T, N, K]     keys/queries, one row per (b, t, n)
 *   v      [B, T, N, V]
 *   a      [B, T, N]        gate logits a_{t,n} = (W_f x_t)_n
 *   alpha  [N], beta [N]    gate parameters (float32); alpha_n >= 0 keeps f in [0, 1]
 *   W      [N, V, V]        per-head transition, right-multiplied:
 *                           (H W)_{ij} = sum_l H_{il} W_{lj}
 *   w_r    [N, V]           value residual weight (float32)
 *   H0     [B, N, K, V]     initial state (float32), or NULL for zeros
 *   y      [B, T, N, V]     readout (float32), written
 *   H_T    [B, N, K, V]     final state (float32), written unless NULL
 *
 * Ownership and threading.  The caller owns every buffer: device pointers
 * (cudaMalloc'd or torch-owned) valid until the work on `stream` completes.
 * The library allocates no device memory per call, keeps no per-call state, and
 * only enqueues work on `stream` (a cudaStream_t passed as void*; NULL is the
 * legacy default stream); it returns before the GPU finishes.  Calls from
 * several host threads are safe.  H0 == H_T (in place) is allowed: each pair's
 * initial state is read before anything of that pair's final state is written.
 * No other output may alias an input.
 *
 * Errors.  Arguments are validated on the host before anything is enqueued;
 * a failed check returns an error and launches nothing.  A bounded device-side
 * wait that gives up is recorded in a per-device status word and reported by
 * m2rnn_stream_status().  The kernels never trap.
 */
#ifndef M2RNN_H
#define M2RNN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum m2rnn_status {
  M2RNN_OK = 0,
  M2RNN_ERR_INVALID_ARG = 1,   /* null required pointer, B/N/K/V < 1, T < 0, misaligned pointer */
  M2RNN_ERR_UNSUPPORTED = 2,   /* shape outside what the selected path supports */
  M2RNN_ERR_CUDA = 3,          /* a CUDA runtime call or launch failed */
  M2RNN_ERR_TIMEOUT = 4        /* a bounded device wait gave up (from m2rnn_stream_status) */
} m2rnn_status;

/*
 * fp32-operand path.  Every tensor is float32.  Supports 1 <= K, V <= 128 and
 * any B, N >= 1, T >= 0.  tanh, exp and log1p are the accurate CUDA math
 * functions; the contraction H W is an fp32 dot product.
 * T == 0 writes H_T = H0 (or zeros) and no y.
 * Returns INVALID_ARG for a null alpha/beta/W/w_r pointer, a null q/k/v/a/y
 * pointer when T > 0 (the empty tensors of T == 0 may be NULL), B, N, K, V < 1
 * or T < 0; UNSUPPORTED for K or V > 128; CUDA if the launch fails.
 */
m2rnn_status m2rnn_forward_f32(const float* q, const float* k, const float* v, const float* a,
                               const float* alpha, const float* beta, const float* W,
                               const float* w_r, const float* H0, float* y, float* H_T,
                               int B, int T, int N, int K, int V, void* stream);

/*
 * bf16-operand / fp32-state path.  q, k, v, a and W are bfloat16 (passed as
 * their uint16_t bit patterns); alpha, beta, w_r, H0, y and H_T are float32.
 * The state H is carried in fp32 and rounded to bf16 only as the tensor-core
 * operand of each step's H W; the rank-1 term, tanh and gate lerp are fp32, and
 * the readout H_t^T q_t accumulates in fp32 (the eight-row kernels take it on the
 * tensor cores from the same bf16 rounding of H_t that the next step's H W reads).  Supports any 1 <= K <= 128 and V a multiple of 16 with 16 <= V <= 128.
 * K that is not a multiple of 16 runs with its rows padded to the next multiple
 * of 16 inside the kernel (padding rows hold zero state, k and q, stay zero for
 * every t and are never stored), so the results are those of the K-row problem.
 * q, k, v, W, y, H0 and H_T must be 16-byte aligned (INVALID_ARG otherwise).
 * Same argument rules and errors as m2rnn_forward_f32, plus UNSUPPORTED for K or
 * V > 128 and for V not a multiple of 16.
 */
m2rnn_status m2rnn_forward_bf16(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                const uint16_t* a, const float* alpha, const float* beta,
                                const uint16_t* W, const float* w_r, const float* H0, float* y,
                                float* H_T, int B, int T, int N, int K, int V, void* stream);

/*
 * As m2rnn_forward_bf16, with an explicit kernel variant (for testing each
 * variant's parity and for measurement).  variant 0 = automatic choice (what
 * m2rnn_forward_bf16 uses); other values are listed by m2rnn_variant_name().
 * Returns UNSUPPORTED if the variant cannot run this shape.
 */
m2rnn_status m2rnn_forward_bf16_variant(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                        const uint16_t* a, const float* alpha, const float* beta,
                                        const uint16_t* W, const float* w_r, const float* H0,
                                        float* y, float* H_T, int B, int T, int N, int K, int V,
                                        int variant, void* stream);

/*
 * Multi-value sharing (the notes' Sec. 2.4: one query/key set shared by all value
 * heads, N_q = N_k = 1, while each head keeps its own v, f, W and state).  As
 * m2rnn_forward_f32 / m2rnn_forward_bf16_variant, with q and k of shape
 * [B, T, Nqk, K]: Nqk == N gives one query/key vector per head (the plain entry
 * points), Nqk == 1 uses the same q_t, k_t for every head n.  Any other Nqk
 * returns INVALID_ARG.  Input bytes per token-head drop to about 2 (V + 1) + 4K/N
 * on the bf16 path when Nqk == 1.
 */
m2rnn_status m2rnn_forward_f32_qk(const float* q, const float* k, const float* v, const float* a,
                                  const float* alpha, const float* beta, const float* W,
                                  const float* w_r, const float* H0, float* y, float* H_T, int B,
                                  int T, int N, int Nqk, int K, int V, void* stream);
m2rnn_status m2rnn_forward_bf16_qk(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                   const uint16_t* a, const float* alpha, const float* beta,
                                   const uint16_t* W, const float* w_r, const float* H0, float* y,
                                   float* H_T, int B, int T, int N, int Nqk, int K, int V,
                                   int variant, void* stream);

/*
 * Training support (the notes' Sec. 2.6-2.7).  The backward pass re-runs the
 * recurrence while keeping every step's state in HBM, then scans time in reverse.
 *
 * m2rnn_forward_train_*: the forward pass of m2rnn_forward_*_qk that also writes
 *   Hs     [B, N, T, K, V]  Hs[b][n][t] = H_t after step t (t = 0..T-1), the states
 *                           the backward reads.  fp32 entry: float32.  bf16 entry:
 *                           bfloat16 (uint16_t bits), the round-to-nearest-even
 *                           rounding of H_t, i.e. exactly the tensor-core operand
 *                           the next step multiplies by W (B·N·T·K·V·2 bytes).
 *   Hs is required when T > 0 (16-byte aligned on the bf16 entry).  The bf16 entry
 *   runs the state-keeping form of a forward kernel, with that kernel's arithmetic:
 *   the pipelined warp-MMA kernel for K a multiple of 16 up to 64 with V in
 *   {16, 32, 64}; the tcgen05 kernel for K = V = 128; eight SMs per pair (or the
 *   4-CTA cluster kernel when their clusters do not all fit) for K = 64, V = 128;
 *   and the row-warp kernel for every other 1 <= K <= 128 with V a multiple of 16
 *   up to 128 (UNSUPPORTED otherwise).  The fp32 entry supports 1 <= K, V <= 128.
 */
m2rnn_status m2rnn_forward_train_f32(const float* q, const float* k, const float* v,
                                     const float* a, const float* alpha, const float* beta,
                                     const float* W, const float* w_r, const float* H0, float* y,
                                     float* H_T, float* Hs, int B, int T, int N, int Nqk, int K,
                                     int V, void* stream);
m2rnn_status m2rnn_forward_train_bf16(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                      const uint16_t* a, const float* alpha, const float* beta,
                                      const uint16_t* W, const float* w_r, const float* H0,
                                      float* y, float* H_T, uint16_t* Hs, int B, int T, int N,
                                      int Nqk, int K, int V, void* stream);

/*
 * Bytes of device workspace m2rnn_backward_* needs for these sizes (0 for an
 * invalid shape).  Per (b, n) pair it holds the running state gradient and the
 * pair's partial sums of dW, dw_r, dalpha, dbeta; with Nqk == 1 < N also the
 * per-head dq, dk before they are summed over heads.
 */
size_t m2rnn_backward_workspace_bytes(int B, int T, int N, int Nqk, int K, int V);

/*
 * Backward pass: gradients of a loss L that depends on y (dy = dL/dy) and on the
 * final state (dH_T = dL/dH_T, NULL for zero), given the inputs of the forward and
 * its kept states Hs (from m2rnn_forward_train_*, same inputs).  The reverse scan
 * is the notes' Sec. 2.7 with u_t = dy_t, C_T = dH_T:
 *   R_t = C_t + q_t u_t^T,  D_t = ((1 - f_t) R_t) ⊙ (1 - Z_t ⊙ Z_t),
 *   C_{t-1} = f_t R_t + D_t W^T,  dL/df_t = <R_t, H_{t-1} - Z_t>,
 *   dW = sum over b, t of H_{t-1}^T D_t,  dk_t = D_t v_t,
 *   dv_t = D_t^T k_t + w_r ⊙ u_t,  dq_t = H_t u_t,  dH0 = C_{-1},
 * with Z_t = tanh(H_{t-1} W + k_t v_t^T) recomputed from Hs, and the gate of
 * Eq. (13)/(17) differentiated (x = a + beta):
 *   da_t = dL/df_t · (-alpha f sigmoid(x)),  dalpha = sum dL/df_t · (-f softplus(x)),
 *   dbeta = sum da_t,  dw_r = sum over b, t of u_t ⊙ v_t.
 * Outputs (float32, written, caller-owned):
 *   dq, dk [B, T, Nqk, K]  (summed over heads when Nqk == 1)
 *   dv [B, T, N, V], da [B, T, N], dalpha [N], dbeta [N], dW [N, V, V], dw_r [N, V],
 *   dH0 [B, N, K, V] (not written when NULL).
 * dy [B, T, N, V] is float32; Hs has the dtype its forward entry wrote (float32 on
 * the fp32 entry, bf16 bits on the bf16 entry).  On the bf16 entry, t = 0 uses the
 * bf16 rounding of H0, as the forward's first step did.  `workspace` is caller-owned device memory of at least
 * m2rnn_backward_workspace_bytes(...) bytes (INVALID_ARG otherwise); it is
 * overwritten, so two calls in flight at once need two workspaces.  Sums over the
 * batch run in a fixed order: results are deterministic.
 * Errors: INVALID_ARG for a null required pointer (q, k, v, a, Hs, dy, dq, dk, dv,
 * da are required only when T > 0) or a bad size; UNSUPPORTED for K or V > 128.
 * The bf16 entry takes bf16 q, k, v, a, W; its `variant` is 0 (automatic: 5 when
 * K = V = 64 and T > 0, 7 when V = 128, K is a multiple of 16 up to 64 and T > 0,
 * 6 when V = 128, K is a multiple of 16 above 64 and T > 0, else 1),
 * 1 (SIMT kernel, fp32 arithmetic, any K, V <= 128),
 * 2 (H_{t-1} W, D_t W^T and H_{t-1}^T D_t as bf16 warp MMAs with fp32 accumulation) or
 * 3 (H_{t-1} W and H_{t-1}^T D_t on the 5th-generation tensor cores with tensor-memory
 * accumulators, D_t W^T as warp MMAs), 4 (variant 3 with eight compute warps) or 5 (all
 * three products on the 5th-generation tensor cores, the chain product D_t W^T included)
 * or 6 (V = 128: every product on the 5th-generation tensor cores, rows padded to 128;
 * D_t enters the products, dk and dv included, rounded to bf16) or 7 (variant 6 with the
 * recurrence's products transposed, so that the tensor-memory lanes run over the 128
 * columns and no row is padding; K <= 64).
 * Variants 2 to 5 need K = V = 64, variant 6 V = 128 and K a multiple of 16, variant 7
 * V = 128 and K a multiple of 16 up to 64 (UNSUPPORTED otherwise); all of them need q, k, v, W, Hs, dy, dv, H0, dH_T, dH0
 * 16-byte aligned.  Bits 8 and up
 * of `variant` are test hooks (0).
 */
m2rnn_status m2rnn_backward_f32(const float* q, const float* k, const float* v, const float* a,
                                const float* alpha, const float* beta, const float* W,
                                const float* w_r, const float* H0, const float* Hs,
                                const float* dy, const float* dH_T, float* dq, float* dk,
                                float* dv, float* da, float* dalpha, float* dbeta, float* dW,
                                float* dw_r, float* dH0, int B, int T, int N, int Nqk, int K,
                                int V, void* workspace, size_t workspace_bytes, void* stream);
m2rnn_status m2rnn_backward_bf16(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                 const uint16_t* a, const float* alpha, const float* beta,
                                 const uint16_t* W, const float* w_r, const float* H0,
                                 const uint16_t* Hs, const float* dy, const float* dH_T, float* dq,
                                 float* dk, float* dv, float* da, float* dalpha, float* dbeta,
                                 float* dW, float* dw_r, float* dH0, int B, int T, int N, int Nqk,
                                 int K, int V, int variant, void* workspace,
                                 size_t workspace_bytes, void* stream);

/*
 * m2rnn_backward_bf16 without a caller workspace: the workspace comes from a fixed
 * 16 MiB scratch array inside the library (one per device).  The M²RNN notes have
 * no counterpart to this entry point; it computes exactly what m2rnn_backward_bf16
 * (variant 0) computes.
 *   * Shapes whose workspace (m2rnn_backward_workspace_bytes) exceeds 16 MiB return
 *     UNSUPPORTED before anything is enqueued; no memory is ever allocated.
 *   * Every call on a device shares its scratch: calls whose work could overlap in
 *     time (other streams or host threads, unordered) race and give wrong results.
 *     Order them on one stream or with events.
 *   * The first call on a device resolves the scratch address (it may load the
 *     module); make that first call before capturing a stream into a CUDA graph.
 *     The address is cached per CUDA context: after a cudaDeviceReset the next call
 *     resolves it again (and must, again, come before any capture).
 */
m2rnn_status m2rnn_backward_bf16_noalloc(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                         const uint16_t* a, const float* alpha, const float* beta,
                                         const uint16_t* W, const float* w_r, const float* H0,
                                         const uint16_t* Hs, const float* dy, const float* dH_T,
                                         float* dq, float* dk, float* dv, float* da, float* dalpha,
                                         float* dbeta, float* dW, float* dw_r, float* dH0, int B,
                                         int T, int N, int Nqk, int K, int V, void* stream);

/*
 * One decode step (T = 1) for serving with a fixed-size state: the forward pass of a
 * single token per (b, n), state in, state out.
 *   q, k   [B, Nqk, K] bf16 (Nqk == N, or 1 shared by all heads)
 *   v      [B, N, V] bf16,  a [B, N] bf16
 *   H_in   [B, N, K, V] float32 state before the token (NULL: zero state)
 *   H_out  [B, N, K, V] float32 state after the token (required; H_out == H_in updates
 *          the state in place)
 *   y      [B, N, V] float32
 * The arithmetic is exactly one step of m2rnn_forward_bf16's warp-MMA kernels
 * (the pipelined kernel and the row-warp kernel), so T successive calls reproduce a
 * T-step forward on those kernels bit for bit.  K = V = 128 and K = 64, V = 128 run
 * the forward on other kernels (other summation orders): there the results agree
 * within the bf16 path's tolerance, not bit for bit.  Small batches run one block per (b, n) pair;
 * K = V = 64 with at least 2048 pairs (and every tensor 16-byte aligned) runs a
 * persistent kernel that streams each pair's state and W through shared memory with TMA
 * (same arithmetic, same bits; its bounded waits report timeouts through
 * m2rnn_stream_status).  Either launch is a single kernel, suitable for CUDA-graph capture.
 * Supports any 1 <= K <= 128 and V a multiple of 16 with 16 <= V <= 128 (UNSUPPORTED
 * otherwise; K that is not a multiple of 16 is padded with zero rows as in
 * m2rnn_forward_bf16).  Same pointer and size errors as m2rnn_forward_bf16 (INVALID_ARG
 * for a null H_out, or W not 16-byte aligned).
 */
m2rnn_status m2rnn_decode_step_bf16(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                    const uint16_t* a, const float* alpha, const float* beta,
                                    const uint16_t* W, const float* w_r, const float* H_in,
                                    float* H_out, float* y, int B, int N, int Nqk, int K, int V,
                                    void* stream);

/*
 * As m2rnn_decode_step_bf16 with an explicit kernel: variant 0 = automatic (what
 * m2rnn_decode_step_bf16 uses), 1 = one block per (b, n) pair, 2 = the persistent
 * TMA-fed kernel at any pair count (K = V = 64 and every tensor 16-byte aligned, else
 * UNSUPPORTED).  Both give the same bits.  Bits 8 and up of `variant` are test hooks
 * (0); they act on the persistent kernel only (the per-pair kernel has no device waits).
 * Any other low byte returns INVALID_ARG.
 */
m2rnn_status m2rnn_decode_step_bf16_variant(const uint16_t* q, const uint16_t* k,
                                            const uint16_t* v, const uint16_t* a,
                                            const float* alpha, const float* beta,
                                            const uint16_t* W, const float* w_r,
                                            const float* H_in, float* H_out, float* y, int B,
                                            int N, int Nqk, int K, int V, int variant,
                                            void* stream);

/*
 * The block's elementwise stages around the recurrence (the notes' Sec. 2.3,
 * Eq. (14)-(23); the projections W_q, W_k, W_v, W_g, W_f, W_o are plain GEMMs outside).
 *
 * m2rnn_conv_silu_bf16: prologue of q, k and v (call once per tensor).
 *   out[b,t,c] = SiLU(bias[c] + sum_{j=0..3} w[c][j] * x[b, t-3+j, c]),  x[b, t<0, c] = 0
 *   x, out [B, T, C] bf16 (16-byte aligned, C % 8 == 0, else UNSUPPORTED; out must not
 *   overlap x); w [C, 4] float32 (16-byte aligned); bias [C] float32 or NULL (none).
 *   Its output, viewed as [B, T, N, K] or [B, T, N, V], is the recurrence's q, k or v.
 *
 * m2rnn_gate_rmsnorm_bf16: epilogue.  For each of `rows` rows of D values (a token's
 *   readout over all heads, D = N V, the recurrence's y viewed as [B T, D]):
 *   z = y ⊙ SiLU(g_pre),  out = w_norm ⊙ z / sqrt(mean(z^2) + eps)
 *   (output gate first, then RMSNorm over the whole token).  y float32, g_pre and out
 *   bf16, w_norm [D] float32, eps >= 0; all 16-byte aligned; D % 8 == 0 (else
 *   UNSUPPORTED).  out is ready to be the W_o GEMM's operand.
 * Both: fp32 arithmetic, results rounded to bf16 (nearest even); memory-bound, every
 * element read and written once.
 */
m2rnn_status m2rnn_conv_silu_bf16(const uint16_t* x, const float* w, const float* bias,
                                  uint16_t* out, int B, int T, int C, void* stream);
m2rnn_status m2rnn_gate_rmsnorm_bf16(const float* y, const uint16_t* g_pre, const float* w_norm,
                                     float eps, uint16_t* out, long long rows, int D,
                                     void* stream);

/*
 * The block prologue fused into the bf16 forward (the notes' Sec. 2.3, Eq. (14)-(16)): the
 * recurrence of m2rnn_forward_bf16_qk on
 *   q = SiLU(conv(xq)), k = SiLU(conv(xk)), v = SiLU(conv(xv)),
 * each a causal depthwise conv of kernel 4 along t exactly as m2rnn_conv_silu_bf16 computes
 * it (same fp32 operations, the result rounded to bf16), so y and H_T are bit-identical to
 * m2rnn_conv_silu_bf16 on each projection followed by m2rnn_forward_bf16_qk.  The convolved
 * q, k, v are never written to memory.
 *   xq, xk  [B, T, Nqk, K] bf16, raw projections; conv taps wq, wk [Nqk*K][4] float32
 *   xv      [B, T, N, V] bf16; taps wv [N*V][4]
 *   bq, bk, bv: biases [Nqk*K] / [N*V] float32, or NULL for zero
 * Other arguments and errors as m2rnn_forward_bf16_qk, plus INVALID_ARG for a null tap
 * pointer (T > 0) or taps not 16-byte aligned.  Runs on the eight-row kernels, so it takes
 * K in {32, 64} and V in {16, 32, 48, 64} (UNSUPPORTED otherwise).  It saves the memory and
 * traffic of the convolved q, k, v but not time: on GB300 it runs slower than the separate
 * prologue plus forward (6.49 ms against 0.37 + 4.26 ms at B=8, T=16384, N=16, K=V=64).
 */
m2rnn_status m2rnn_forward_conv_bf16(const uint16_t* xq, const uint16_t* xk, const uint16_t* xv,
                                     const float* wq, const float* bq, const float* wk,
                                     const float* bk, const float* wv, const float* bv,
                                     const uint16_t* a, const float* alpha, const float* beta,
                                     const uint16_t* W, const float* w_r, const float* H0,
                                     float* y, float* H_T, int B, int T, int N, int Nqk, int K,
                                     int V, void* stream);

/*
 * The selective state space block: what lies between its projections.  The linear
 * counterpart of the M²RNN recurrence on the same tensors (the gate of Eq. (13)/(17) with
 * the step size d_t in front of the outer product, no tanh and no W), with the short causal
 * convolution in front of it and the gated group norm behind it, each for prompts, single
 * tokens and training.  Not part of the notes' block; hybrid stacks (the notes' Sec. 5.2)
 * alternate such layers with M²RNN layers.
 *
 * Strides.  Where an entry takes strides they are in elements; a token's channels (heads
 * and their width) are contiguous, so slices of a wider projection or conv output can be
 * passed without a copy.  All other tensors are dense.
 *
 * Sizes.  Tensors may hold more than 2^31 values; T <= 2^31 - 128, and B C (conv), B N
 * (scan) < 2^31.  The backwards count their sums in 32 bits: 5 C and 2 D (norm) and
 * N (2 + V) <= 2^31 - 32.  UNSUPPORTED above.
 *
 * m2rnn_conv_silu_window_bf16: m2rnn_conv_silu_bf16 continuing an earlier call.
 *   out[b,t,c] = SiLU(bias[c] + sum_{j=0..3} w[c][j] * X[b, t-3+j, c])
 *   with X[b, -3..-1] = window_in[b] (NULL: zeros) and X[b, t >= 0] = x[b, t].
 *   x [B, T, C] bf16 with strides (x_batch, x_token); window_in, window_out [B, 3, C] bf16:
 *   the last three inputs, oldest first (window_out NULL: not written; window_out ==
 *   window_in updates in place); out [B, T, C] bf16 dense; w [C, 4] float32 (16-byte
 *   aligned, else INVALID_ARG); bias [C] float32 or NULL (none).  T = 1 is the single-token
 *   form.  T = 0 copies the window.  Any C >= 1; rows of C % 4 == 0 channels with every bf16
 *   pointer and stride 8-byte aligned run on 8-byte accesses.
 * m2rnn_conv_silu_backward_bf16: its gradients, given dout [B, T, C] bf16 (dense):
 *   dx [B, T, C] bf16 (dense), dw [C, 4], dbias [C] float32 (NULL: not written),
 *   dwindow [B, 3, C] bf16 (NULL: not written).  The workspace (16-byte aligned, at least
 *   m2rnn_conv_silu_backward_workspace_bytes) holds partial sums, added in a fixed order.
 */
m2rnn_status m2rnn_conv_silu_window_bf16(const uint16_t* x, const float* w, const float* bias,
                                         const uint16_t* window_in, uint16_t* out,
                                         uint16_t* window_out, int B, int T, int C,
                                         long long x_batch, long long x_token, void* stream);
size_t m2rnn_conv_silu_backward_workspace_bytes(int B, int T, int C);
m2rnn_status m2rnn_conv_silu_backward_bf16(const uint16_t* x, const float* w, const float* bias,
                                           const uint16_t* window_in, const uint16_t* dout,
                                           uint16_t* dx, float* dw, float* dbias,
                                           uint16_t* dwindow, int B, int T, int C,
                                           long long x_batch, long long x_token, void* workspace,
                                           size_t workspace_bytes, void* stream);

/*
 * The selective scan.  For every (batch b, head n), with x_t = a_{t,n} + beta_n:
 *   d_t = softplus(x_t),  f_t = exp(-alpha_n d_t)
 *   H_t = f_t H_{t-1} + d_t k_t v_t^T,   y_t = H_t^T q_t + w_r ⊙ v_t
 *   q, k  [B, T, Nqk, K] bf16, Nqk >= 1 dividing N: head n reads head n Nqk / N of q and k
 *   v     [B, T, N, V], a [B, T, N] bf16;  alpha, beta [N], w_r [N, V] float32
 *   H0, H_T [B, N, K, V] float32 (NULL: zeros / not written; H_T == H0 is allowed)
 *   y     [B, T, N, V] bf16, dense
 *   strides: eight values, (batch, token) of q, k, v and a in turn, or NULL for dense.
 * 1 <= K, V <= 128 (UNSUPPORTED above), B, N >= 1, T >= 0.  a = -infinity makes a token
 * inert (d = 0, f = 1); a token with a large enough a resets the state (f = 0).
 * The state and every sum are float32; the operands of the tensor-core products are bf16.
 * q, k, v (and dy below) have to be finite: tokens are taken in chunks of 128 and what lies
 * behind the causal mask is multiplied by zero, so an infinity or NaN reaches every token of
 * its chunk, earlier ones too, and all later ones.  Operands of K, V % 8 == 0 values with
 * 16-byte aligned pointers and strides are loaded in tiles; any others value by value, slowly.
 * m2rnn_ssm_forward_bf16 with Hs != NULL also keeps what the backward reads:
 *   Hs    m2rnn_ssm_states_bytes(...) bytes, 16-byte aligned: the state before every chunk
 *         of 128 tokens and the final one, each value as the sum of two bf16 values.
 * The workspace (16-byte aligned, at least m2rnn_ssm_workspace_bytes(..., 0) for the
 * forward and (..., 1) for the backward; NULL where that is 0) is overwritten: calls in
 * flight at once need one each.
 */
size_t m2rnn_ssm_states_bytes(int B, int T, int N, int K, int V);
size_t m2rnn_ssm_workspace_bytes(int B, int T, int N, int Nqk, int K, int V, int backward);
m2rnn_status m2rnn_ssm_forward_bf16(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                    const uint16_t* a, const float* alpha, const float* beta,
                                    const float* w_r, const float* H0, uint16_t* y, float* H_T,
                                    void* Hs, const long long* strides, int B, int T, int N,
                                    int Nqk, int K, int V, void* workspace,
                                    size_t workspace_bytes, void* stream);
/*
 * Gradients of a loss through y (dy [B, T, N, V] bf16, dense) and H_T (dH_T [B, N, K, V]
 * float32, NULL: zero), from the forward's inputs and its Hs.  With G the gradient of H_t,
 * G_t = f_{t+1} G_{t+1} + q_t dy_t^T, and g_t = f_t <G_t, H_{t-1}>:
 *   dq_t = H_t dy_t, dk_t = d_t G_t v_t, dv_t = d_t G_t^T k_t + w_r ⊙ dy_t,
 *   da_t = sigmoid(x_t) (k_t^T G_t v_t - alpha g_t),
 *   dalpha = -sum d_t g_t, dbeta = sum da_t, dw_r = sum dy_t ⊙ v_t, dH0 = f_1 G_1.
 * dq, dk [B, T, Nqk, K] (summed over the heads that share them), dv [B, T, N, V],
 * da [B, T, N]: bf16, dense; dalpha, dbeta [N], dw_r [N, V], dH0 [B, N, K, V] (NULL: not
 * written): float32.  Sums run in a fixed order.
 */
m2rnn_status m2rnn_ssm_backward_bf16(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                     const uint16_t* a, const float* alpha, const float* beta,
                                     const float* w_r, const void* Hs, const uint16_t* dy,
                                     const float* dH_T, uint16_t* dq, uint16_t* dk, uint16_t* dv,
                                     uint16_t* da, float* dalpha, float* dbeta, float* dw_r,
                                     float* dH0, const long long* strides, int B, int T, int N,
                                     int Nqk, int K, int V, void* workspace,
                                     size_t workspace_bytes, void* stream);
/*
 * One token (T = 1): q, k [B, Nqk, K], v [B, N, V], a [B, N] bf16 dense, H_in, H_out
 * [B, N, K, V] float32 (H_in NULL: zeros; H_out == H_in updates in place), y [B, N, V] bf16.
 * fp32 arithmetic throughout.
 */
m2rnn_status m2rnn_ssm_step_bf16(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                 const uint16_t* a, const float* alpha, const float* beta,
                                 const float* w_r, const float* H_in, float* H_out, uint16_t* y,
                                 int B, int N, int Nqk, int K, int V, void* stream);

/*
 * Gated group norm over the channels of one token: each of `rows` rows of D values is cut
 * into `groups` groups of E = D / groups consecutive channels,
 *   n = (y - mean) / sqrt(var + eps)  (mean and biased variance of the group),
 *   p = w ⊙ n + bias,   out = p ⊙ SiLU(g_pre), or SiLU(p) where g_pre is NULL.
 * y [rows, D] float32 (y_f32 != 0) or bf16; g_pre, out bf16; w, bias [D] float32 (bias
 * NULL: none).  E <= 8192 (UNSUPPORTED above; INVALID_ARG where groups does not divide D
 * or eps < 0).  A group is read once and kept in registers; E % 8 == 0 with 16-byte aligned
 * pointers runs on 16-byte accesses.
 * Backward: dout bf16 -> dy (of y's type), dg_pre bf16 (with g_pre), dw, dbias [D] float32
 * (dbias NULL: not written), with a workspace for partial sums added in a fixed order.
 */
m2rnn_status m2rnn_gate_groupnorm(const void* y, int y_f32, const uint16_t* g_pre, const float* w,
                                  const float* bias, float eps, uint16_t* out, long long rows,
                                  int D, int groups, void* stream);
size_t m2rnn_gate_groupnorm_backward_workspace_bytes(long long rows, int D, int groups);
m2rnn_status m2rnn_gate_groupnorm_backward(const void* y, int y_f32, const uint16_t* g_pre,
                                           const float* w, const float* bias, float eps,
                                           const uint16_t* dout, void* dy, uint16_t* dg_pre,
                                           float* dw, float* dbias, long long rows, int D,
                                           int groups, void* workspace, size_t workspace_bytes,
                                           void* stream);

/*
 * What stands around a block in a stack: the residual's addition with the RMS norm in front of a
 * block, the projections in 8 bits, and the clipping of a training step's gradients.
 *
 * Residual RMS norm.  Each of `rows` rows of D channels:
 *   h = stream_in + x  (rounded to the stream's type; x NULL: h = stream_in)
 *   out = h / sqrt(mean(h^2) + eps) ⊙ w
 * x bf16; stream_in and h bf16 or float32 (stream_f32 != 0); w [D] float32.  x_row and stream_row are the
 * elements from one row to the next; h and out [rows, D] are dense.  h may be NULL without x (not written)
 * and may be stream_in itself (in place) where that is dense.  The norm is taken of the rounded h, in
 * float32: |h| above 1e19 overflows its square (out is 0 there), and with eps = 0 a row whose values are all below
 * 1e-19 loses digits of their squares.  D <= 16384 (UNSUPPORTED above).
 * A NaN gives NaN in all of its row, an infinity in its channel (in 8 bits in its 128) and zeros in the rest of
 * the row; other rows are untouched.  16-byte aligned pointers run on 16-byte accesses where D % 8 == 0 and rows
 * are aligned so, or where the rows' distances are D or a multiple of 8 more.  The order of a row's sum depends on
 * the sizes and alignment of the call and, where D % 8 != 0, on the row's place; the same call gives the same bits.
 * m2rnn_add_rmsnorm: out bf16.  m2rnn_add_rmsnorm_fp8: out in 8 bits (see below), q [rows, D] with q_row
 *   bytes from row to row (q and q_row multiples of 16) and scales [rows, ceil(D / 128)], dense.
 * m2rnn_add_rmsnorm_backward: with dout [rows, D] bf16 and dh [rows, D] of the stream's type (the gradient
 *   that reaches h by the stream; NULL: none), g = dout ⊙ w and r = 1 / sqrt(mean(h^2) + eps):
 *     d = dh + r g - h r^3 mean(g ⊙ h),   dw = sum over rows of dout ⊙ h r
 *   dx (bf16) and dresidual (of the stream's type) are both d; either may be NULL, not both.  dx or
 *   dresidual may be dh itself where the types agree.  All dense.  The workspace (16-byte aligned) holds
 *   partial sums, added in a fixed order.
 */
m2rnn_status m2rnn_add_rmsnorm(const uint16_t* x, long long x_row, const void* stream_in,
                               int stream_f32, long long stream_row, const float* w, float eps,
                               void* h, uint16_t* out, long long rows, int D, void* stream);
m2rnn_status m2rnn_add_rmsnorm_fp8(const uint16_t* x, long long x_row, const void* stream_in,
                                   int stream_f32, long long stream_row, const float* w, float eps,
                                   void* h, uint8_t* q, long long q_row, uint8_t* scales,
                                   long long rows, int D, void* stream);
size_t m2rnn_add_rmsnorm_backward_workspace_bytes(long long rows, int D);
m2rnn_status m2rnn_add_rmsnorm_backward(const void* h, int stream_f32, const float* w, float eps,
                                        const uint16_t* dout, const void* dh, uint16_t* dx,
                                        void* dresidual, float* dw, long long rows, int D,
                                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * 8 bits: e4m3 values q and, for each 128 consecutive values of a row (the last block may be shorter), one
 * scale s, a power of two kept as its exponent plus 127 in a byte (e8m0); a value stands for q s.  s is the
 * least power of two with max |value| / s <= 448, 2^-126 at the least; q is value / s rounded to the
 * nearest, ties to even.  A block that holds an infinity or a NaN gets the scale NaN (255) and NaNs.
 * Rows start q_row bytes apart; q and q_row are multiples of 16.  Scales are dense.
 * m2rnn_quantise_fp8: x [rows, D] bf16 or float32 (x_f32 != 0), x_row elements from row to row ->
 *   q [rows, D], scales [rows, ceil(D / 128)].
 * m2rnn_quantise_weight_fp8: w [N, K], one scale for each 128 x 128 block -> q [N, K],
 *   scales [ceil(N / 128), ceil(K / 128)].
 * m2rnn_linear_fp8: out[m, n] = sum_k x[m, k] w[n, k] of such values, x [M, K] with a scale for each 128
 *   of a row, w [N, K] with one for each 128 x 128 block; out [M, N] bf16 or float32 (out_f32 != 0), dense.
 *   Sums are float32 on the tensor cores.  A NaN of x spoils its row of out, one of w its column; a scale
 *   of w that is NaN spoils the columns of its block.  A form for serving: it has no gradient.  Fastest with
 *   rows of x and w on 128-byte boundaries and rows of out that are whole multiples of 32 bytes at a 32-byte
 *   aligned address.
 * m2rnn_linear_quantise_fp8: the same with x [M, K] bf16 or float32 (x_f32 != 0), x_row elements from row to
 *   row, as m2rnn_quantise_fp8 makes it 8 bits; up to 16 rows of bf16 within the product's own launch.  The
 *   workspace (16-byte aligned; NULL where its size is 0) is overwritten.
 */
m2rnn_status m2rnn_quantise_fp8(const void* x, int x_f32, long long x_row, uint8_t* q,
                                long long q_row, uint8_t* scales, long long rows, int D,
                                void* stream);
m2rnn_status m2rnn_quantise_weight_fp8(const void* w, int w_f32, long long w_row, uint8_t* q,
                                       long long q_row, uint8_t* scales, int N, int K,
                                       void* stream);
m2rnn_status m2rnn_linear_fp8(const uint8_t* x, long long x_row, const uint8_t* x_scales,
                              const uint8_t* w, long long w_row, const uint8_t* w_scales, void* out,
                              int out_f32, long long M, int N, int K, void* stream);
size_t m2rnn_linear_quantise_workspace_bytes(int x_f32, long long M, int K);
m2rnn_status m2rnn_linear_quantise_fp8(const void* x, int x_f32, long long x_row, const uint8_t* w,
                                       long long w_row, const uint8_t* w_scales, void* out,
                                       int out_f32, long long M, int N, int K, void* workspace,
                                       size_t workspace_bytes, void* stream);

/*
 * The global norm of `count` gradients, and their clipping:
 *   norm = sqrt(sum of all values squared),   out[i] = grads[i] min(1, max_norm / norm)
 * grads[i] holds values[i] values (0 is allowed), float32 (is_f32[i] != 0) or bf16, anywhere on a
 * boundary of its type; out[i] is grads[i] itself (in place) or memory apart.  These four arrays are host
 * memory, read during the call.  norm: one float32 on the device.  out NULL: the norm alone (max_norm is
 * not read).  Values that hold an infinity or a NaN are not clipped: they stay as they are, and norm says
 * so.  A norm of finite values above float32's range reads as infinite too, but does clip.
 * INVALID_ARG where something that is written shares memory with another gradient or output, or max_norm
 * is negative, infinite or NaN; UNSUPPORTED above 2^40 values.  Squares are summed in 64 bits above a few
 * of them, in a fixed order, and also where they leave float32's range.  The workspace (16-byte aligned,
 * at least m2rnn_grad_norm_workspace_bytes) is overwritten.
 */
size_t m2rnn_grad_norm_workspace_bytes(int count);
m2rnn_status m2rnn_clip_grad_norm(const void* const* grads, void* const* out,
                                  const long long* values, const unsigned char* is_f32, int count,
                                  float max_norm, float* norm, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* Name of a bf16 kernel variant (NULL for an unknown id).  Id 0 is "auto". */
const char* m2rnn_variant_name(int variant);

/* The variant m2rnn_forward_bf16 would pick for this shape on the current
 * device (>0), or 0 if no variant supports it. */
int m2rnn_pick_variant(int B, int T, int N, int K, int V);

/* 1 if bf16 kernel variant `variant` (> 0) can run this shape, else 0. */
int m2rnn_variant_supports(int variant, int B, int T, int N, int K, int V);

/*
 * The balanced schedule of the K = V = 128 tensor-core forward (variant
 * "tcgen05_k128_v128_balanced", chosen automatically when there are more
 * (batch, head) pairs than resident thread blocks).  Lay the B*N pairs' steps
 * end to end (pair p = b*N + n owns positions [p*T, (p+1)*T)); stretch `worker`
 * of `workers` (one thread block each) covers positions [*begin, *end).  A pair
 * cut by a boundary runs its
 * first steps at the start of the later block's stretch and its last steps at
 * the end of the earlier block's stretch (at least 129 of them: the handed-over
 * state travels through that pair's own y rows before they are written).
 * Host-only arithmetic, exposed so the schedule can be checked without a GPU.
 * Returns 0, or -1 for pairs, T or workers < 1, or worker outside [0, workers).
 */
int m2rnn_balanced_stretch(long long pairs, int T, long long workers, long long worker,
                           long long* begin, long long* end);

/*
 * Synchronises `stream`, then returns and clears the current device's status
 * word: M2RNN_ERR_TIMEOUT if a kernel's bounded wait gave up since the last
 * call, M2RNN_ERR_CUDA if the synchronisation itself failed, else M2RNN_OK.
 */
m2rnn_status m2rnn_stream_status(void* stream);

/* Static, human-readable name of a status code. */
const char* m2rnn_status_string(m2rnn_status s);

/* Library version, major * 10000 + minor * 100 + patch. */
int m2rnn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* M2RNN_H */
