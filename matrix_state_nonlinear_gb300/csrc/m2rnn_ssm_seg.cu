// m2rnn_ssm_seg.cu — the states at which the scan's segments start.
//
// Where there are fewer (batch, head) pairs than SMs, a pair's sequence is cut into segments that
// run side by side.  One launch sums every piece's own state from zero,
//   forward:   sum_s exp(c_end - c_s) d_s k_s v_s^T        (reads k, v)
//   backward:  sum_t exp(c_t) q_t dy_t^T                   (reads q, dy; the state's gradient)
// and a second, element by element, chains the pieces of a pair into the state before each piece
// (or the state's gradient after it).  Pieces are finer than the segments that use them, so that
// the first launch fills the GPU: about three blocks of four warps per SM.
//
// The products are m16n8k16 on bf16, the weight times k (or q) entering as two bf16 values: the
// sums are float32 throughout, 17 bits from each weighted operand.  The traffic of k and v bounds
// the first launch (2 (K + V) bytes a token and head against 4 K V tensor operations).
#include <mutex>

#include "m2rnn_ssm_mma.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 128;
constexpr int L = 64;  // tokens per step; pieces are whole chunks
constexpr int kSteps = kSsmChunk / L;
constexpr int VT = kSsmColumns;
constexpr int kStages = 3;

struct alignas(16) Weights {  // of one chunk
  float w[L];
  float total;  // log2 of the chunk's decay
};

template <int KP>
struct Smem {
  static constexpr int kX = L * KP * 2;
  static constexpr int kStage = kX + L * VT * 2;
  static constexpr int kWeights = kStages * kStage;
  static constexpr int kBytes = kWeights + 8 * (int)sizeof(Weights);
};

// Piece `blockIdx.y` of a pair: chunks [piece * per, ...).  x is k and y is v, or, with REVERSE,
// q and dy with the chunks walked backwards.
template <int KP, bool REVERSE>
__global__ void __launch_bounds__(kThreads, KP <= 64 ? 3 : 2)
    ssm_piece_kernel(SegmentProblem p, int per, bool vec) {
  using S = Smem<KP>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = smem_u32(smem);
  Weights* weights = reinterpret_cast<Weights*>(smem + S::kWeights);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c2 = (lane & 3) * 2;
  const int vtiles = (p.V + VT - 1) / VT;
  const int vt = blockIdx.x % vtiles, piece = blockIdx.y + (REVERSE ? 1 : 0);
  const long long pair = blockIdx.x / vtiles;
  const int n = (int)(pair % p.N);
  const long long b = pair / p.N;
  const int head = (int)((long long)n * p.Nqk / p.N);
  const int steps = (p.T + L - 1) / L;
  const int first = piece * per * kSteps, count = min(steps, first + per * kSteps) - first;
  const int v0 = vt * VT, vw = min(VT, p.V - v0);
  const uint16_t* ag = p.a + b * p.sa.batch + n;
  const float alpha = p.alpha[n], beta = p.beta[n];
  auto chunk_at = [&](int i) { return REVERSE ? first + count - 1 - i : first + i; };

  TileLoader<KP, L, kThreads> load_x;
  TileLoader<VT, L, kThreads> load_y;
  load_x.init(p.x + b * p.sx.batch + (long long)head * p.K, p.sx.token, p.K, tid);
  load_y.init(p.y + b * p.sy.batch + (long long)n * p.V + v0, p.sy.token, vw, tid);
  auto load = [&](int i) {
    if (i < count) {
      const uint32_t tile = base + i % kStages * S::kStage;
      const int chunk = chunk_at(i), rows = min(L, p.T - chunk * L);
      load_x.load(tile, (long long)chunk * L, rows, vec, tid);
      load_y.load(tile + S::kX, (long long)chunk * L, rows, vec, tid);
    }
    cp_async_commit();
  };
  // One warp's chunk of the next four: its weights.
  auto put_weights = [&](int i) {
    if (i >= count) return;
    const int t = chunk_at(i) * L + lane;
    const float2 g0 = ssm_gate(t < p.T ? bf16_to_f(ag[t * p.sa.token]) : -INFINITY, alpha, beta);
    const float2 g1 = ssm_gate(t + 32 < p.T ? bf16_to_f(ag[(t + 32) * p.sa.token]) : -INFINITY, alpha, beta);
    const ChunkSums s = chunk_sums(g0.y * kLog2e, g1.y * kLog2e, lane);
    Weights& o = weights[i & 7];
    o.w[lane] = REVERSE ? exp2_approx(s.cum0) : g0.x * exp2_approx(s.rest0);
    o.w[lane + 32] = REVERSE ? exp2_approx(s.cum1) : g1.x * exp2_approx(s.rest1);
    if (lane == 0) o.total = s.total;
  };

  using T = StateTiles<KP, VT>;
  const int m0 = T::row_tile(warp), nt0 = T::col_tile(warp);
  float H[T::MT][T::NT][4];
#pragma unroll
  for (int m = 0; m < T::MT; ++m)
#pragma unroll
    for (int j = 0; j < T::NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) H[m][j][e] = 0.f;
  const uint32_t part_x = lane_part<KP>(lane, false), part_y = lane_part<VT>(lane, true);

  load(0);
  load(1);
  put_weights(warp);
  float decay = 0.f;
  for (int i = 0; i < count; ++i) {
    cp_async_wait<1>();
    __syncthreads();
    load(i + 2);
    const uint32_t tile = base + i % kStages * S::kStage;
    const Weights& w = weights[i & 7];
    decay += w.total;
    scale_state<T>(H, exp2_approx(w.total));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t yf[4][4];
#pragma unroll
      for (int np = 0; np < 4; ++np) ldsm_x4_trans(yf[np], frag_at<VT>(tile + S::kX, part_y, j * 16, np * 2));
      add_outer<KP, T>(H, tile, part_x, w.w, yf, j, m0, nt0, c2);
    }
    if ((i & 3) == 3) put_weights(i + 1 + warp);
  }
  cp_async_wait<0>();
  if (vt == 0 && tid == 0) p.decay[pair * p.pieces + piece] = decay;
  float* dst = p.state + ((size_t)pair * p.pieces + piece) * p.K * p.V;
#pragma unroll
  for (int m = 0; m < T::MT; ++m)
#pragma unroll
    for (int j = 0; j < T::NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = (m0 + m) * 16 + g + (e >> 1) * 8, col = (nt0 + j) * 8 + c2 + (e & 1);
        if (row < p.K && col < vw) dst[(size_t)row * p.V + v0 + col] = H[m][j][e];
      }
}

// state[piece] from the piece's own sum to the state before it (after it, with `reverse`), in
// place: the chain starts at `start` and takes in a piece's decay and sum after it is written.
__global__ void __launch_bounds__(256) ssm_join_kernel(SegmentProblem p, int kv, int reverse) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  const long long pair = blockIdx.y;
  if (i >= kv) return;
  float h = p.start ? p.start[(size_t)pair * kv + i] : 0.f;
  float* s = p.state + (size_t)pair * p.pieces * kv + i;
  const float* d = p.decay + pair * p.pieces;
  constexpr int kAhead = 8;  // pieces loaded at once
  for (int j = 0; j < p.pieces; j += kAhead) {
    float own[kAhead], decay[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (j + u + 1 < p.pieces) {
        const int at = reverse ? p.pieces - 1 - j - u : j + u;
        own[u] = s[(size_t)at * kv];
        decay[u] = d[at];
      }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int at = reverse ? p.pieces - 1 - j - u : j + u;
      if (j + u < p.pieces) s[(size_t)at * kv] = h;
      if (j + u + 1 < p.pieces) h = fmaf(exp2_approx(decay[u]), h, own[u]);
    }
  }
}

template <int KP, bool REVERSE>
cudaError_t run(const SegmentProblem& p, int per, bool vec, cudaStream_t stream) {
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [] {
    attr = cudaFuncSetAttribute(ssm_piece_kernel<KP, REVERSE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Smem<KP>::kBytes);
  });
  if (attr != cudaSuccess) return attr;
  const long long pairs = (long long)p.B * p.N;
  const unsigned units = (unsigned)(pairs * ((p.V + VT - 1) / VT));
  ssm_piece_kernel<KP, REVERSE><<<dim3(units, p.pieces - 1), kThreads, Smem<KP>::kBytes, stream>>>(p, per, vec);
  const int kv = p.K * p.V;
  ssm_join_kernel<<<dim3((kv + 255) / 256, (unsigned)pairs), 256, 0, stream>>>(p, kv, REVERSE);
  return cudaGetLastError();
}

}  // namespace

// Whole segments for every SM at most; segments of at least four chunks.  Pieces: three blocks
// of the first launch per SM, of at least two chunks.
SsmCut ssm_cut(int B, int T, int N, int V) {
  constexpr int kSms = 152;
  const long long units = (long long)B * N * ((V + VT - 1) / VT);
  const int chunks = ssm_chunks(T);
  SsmCut c{1, chunks > 0 ? chunks : 1, 1, chunks > 0 ? chunks : 1};
  long long want = kSms / units;
  if (want > chunks / 4) want = chunks / 4;
  if (want < 2) return c;
  const int per = (int)((chunks + want - 1) / want);
  int fine = (int)(3 * kSms / (units * want));
  if (fine > per / 2) fine = per / 2;
  if (fine < 1) fine = 1;
  c.piece = (per + fine - 1) / fine;
  c.per = c.piece * fine;
  c.fine = fine;
  c.segments = (chunks + c.per - 1) / c.per;
  return c;
}

// Pieces of the whole sequence (the last segment may have fewer than `fine`).
int ssm_pieces(const SsmCut& c, int T) { return (ssm_chunks(T) + c.piece - 1) / c.piece; }

size_t ssm_segment_floats(const SsmCut& c, int B, int T, int N, int K, int V) {
  return c.segments > 1 ? (size_t)B * N * ssm_pieces(c, T) * ((size_t)K * V + 1) : 0;
}

cudaError_t launch_ssm_segments(SegmentProblem p, const SsmCut& c, bool reverse, bool vec, cudaStream_t stream) {
  p.pieces = ssm_pieces(c, p.T);
  p.decay = p.state + (size_t)p.B * p.N * p.pieces * p.K * p.V;
  auto pick = [&](auto rev) {
    constexpr bool R = decltype(rev)::value;
    if (p.K <= 16) return run<16, R>(p, c.piece, vec, stream);
    if (p.K <= 32) return run<32, R>(p, c.piece, vec, stream);
    if (p.K <= 64) return run<64, R>(p, c.piece, vec, stream);
    return run<128, R>(p, c.piece, vec, stream);
  };
  return reverse ? pick(std::true_type{}) : pick(std::false_type{});
}

}  // namespace m2rnn
