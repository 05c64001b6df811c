// m2rnn_ssm_fwd.cu — the selective scan of a prompt in chunks of 64 tokens (see include/m2rnn.h).
//
// With c_t the sum of log f over a chunk up to token t, and H the state before the chunk,
//   y_t = exp(c_t) H^T q_t + sum_{s <= t} exp(c_t - c_s) d_s (q_t . k_s) v_s + w_r v_t
//   H  <- exp(c_63) H + sum_s (exp(c_63 - c_s) d_s k_s) v_s^T
// so that a chunk is five matrix products.  One block of four warps walks the chunks of one
// (batch, head) pair and one tile of 64 value columns; the state stays in float32 registers.
//  * Warp w takes 16 tokens of y (block row rb) and K / 4 rows of the state.  Scores above the
//    diagonal's 16 x 16 block are not computed; so that the warps' unequal work spreads over the
//    SM's four quarters, rb is rotated from block to block.
//  * Scores are decayed in float32 and rounded to bf16 as the operand of the product with v; the
//    state is rounded to bf16 as the operand of H^T q; y is bf16.  The state's own update keeps
//    the float32 weights: weight times k enters as two bf16 values (17 bits), two products.
//  * exp(c_t - c_s) is split at the end of s's block of 16, exp(c_t - c_end) exp(c_end - c_s), two
//    factors of at most one: one exponential per row and block instead of one per score.
//  * Two stages of q, k and v tiles are loaded by cp.async.
// Where the pairs are fewer than the GPU's blocks, the sequence is cut into segments: one launch
// sums each segment's state from zero (k and v only), a second walks the segments of a pair, and
// the main launch starts every segment from its state.
#include <mutex>

#include "m2rnn_ssm_mma.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 128;
constexpr int L = kSsmChunk;
constexpr int VT = 64;  // value columns per block

// Segment cut: segment i covers chunks [i * per, (i + 1) * per).
struct Cut {
  int segments, per;
};

struct alignas(16) Gates {  // of one chunk, per token; read in pairs
  float cum[L];   // log2 of the decay from the chunk's start, the token's own included
  float d[L];     // step size
  float wd[L];    // d times the decay from the token to the end of its 16
  float wk[L];    // d times the decay from the token to the chunk's end
  float total;    // log2 of the whole chunk's decay
};
struct alignas(16) Row {
  float w_r[VT];
};

template <int KP, bool STATES_ONLY>
struct Smem {
  static constexpr int kQ = STATES_ONLY ? 0 : L * KP * 2;
  static constexpr int kK = L * KP * 2;
  static constexpr int kV = L * VT * 2;
  static constexpr int kStage = kQ + kK + kV;
  static constexpr int kH = STATES_ONLY ? 0 : KP * VT * 2;  // the state as bf16, two buffers
  static constexpr int kY = STATES_ONLY || KP >= 64 ? 0 : L * VT * 2;  // y on its way out
  static constexpr int kGates = 2 * kStage + 2 * kH + kY;
  static constexpr int kRow = kGates + 2 * (int)sizeof(Gates);
  static constexpr int kBytes = kRow + (int)sizeof(Row);
  static_assert(kGates % 16 == 0 && sizeof(Gates) % 16 == 0, "pairs of gates are read at once");
};

template <int KP, bool STATES_ONLY>
__global__ void __launch_bounds__(kThreads, KP <= 64 ? 3 : 2)
    ssm_chunk_kernel(SsmProblem p, Cut cut, float* __restrict__ seg_state,
                     float* __restrict__ seg_decay, bool vec) {
  using S = Smem<KP, STATES_ONLY>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = smem_u32(smem);
  Gates* gates = reinterpret_cast<Gates*>(smem + S::kGates);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c2 = (lane & 3) * 2;
  const int vtiles = (p.V + VT - 1) / VT;
  const int vt = blockIdx.x % vtiles, seg = blockIdx.y;
  const long long pair = blockIdx.x / vtiles;
  const int n = (int)(pair % p.N);
  const long long b = pair / p.N;
  const int head = (int)((long long)n * p.Nqk / p.N);
  const int chunks = ssm_chunks(p.T);
  const int first = seg * cut.per, last = min(chunks, first + cut.per);
  const int v0 = vt * VT, vw = min(VT, p.V - v0);  // this block's columns
  const int rb = (warp + blockIdx.x + blockIdx.y) & 3;  // this warp's 16 tokens of y

  const uint16_t* ag = p.a + b * p.sa.batch + n;
  const float alpha = p.alpha[n], beta = p.beta[n];

  auto tile_q = [&](int s) { return base + s * S::kStage; };
  auto tile_k = [&](int s) { return base + s * S::kStage + S::kQ; };
  auto tile_v = [&](int s) { return base + s * S::kStage + S::kQ + S::kK; };
  auto tile_h = [&](int s) { return base + 2 * S::kStage + s * S::kH; };
  TileLoader<KP, L, kThreads> load_q, load_k;
  TileLoader<VT, L, kThreads> load_v;
  if constexpr (!STATES_ONLY) load_q.init(p.q + b * p.sq.batch + (long long)head * p.K, p.sq.token, p.K, tid);
  load_k.init(p.k + b * p.sk.batch + (long long)head * p.K, p.sk.token, p.K, tid);
  load_v.init(p.v + b * p.sv.batch + (long long)n * p.V + v0, p.sv.token, vw, tid);
  auto load_chunk = [&](int chunk, int s) {
    const long long t0 = (long long)chunk * L;
    const int rows = min(L, p.T - chunk * L);
    if constexpr (!STATES_ONLY) load_q.load(tile_q(s), t0, rows, vec, tid);
    load_k.load(tile_k(s), t0, rows, vec, tid);
    load_v.load(tile_v(s), t0, rows, vec, tid);
    cp_async_commit();
  };
  const uint32_t part_k_down = lane_part<KP>(lane, true), part_k_across = lane_part<KP>(lane, false);
  const uint32_t part_v_down = lane_part<VT>(lane, true);
  float* wr = reinterpret_cast<Row*>(smem + S::kRow)->w_r;
  if (!STATES_ONLY && tid < VT) wr[tid] = tid < vw ? p.w_r[(size_t)n * p.V + v0 + tid] : 0.f;
  // The gate logits of a chunk (tokens lane, lane + 32) and what the products need of them.
  auto load_logits = [&](int chunk) {
    const int t = chunk * L + lane;
    float2 a;
    a.x = t < p.T ? bf16_to_f(ag[t * p.sa.token]) : -INFINITY;
    a.y = t + 32 < p.T ? bf16_to_f(ag[(t + 32) * p.sa.token]) : -INFINITY;
    return a;
  };
  auto put_gates = [&](float2 a, int s) {
    const float2 g0 = ssm_gate(a.x, alpha, beta), g1 = ssm_gate(a.y, alpha, beta);
    const ChunkSums sum = chunk_sums(g0.y * kLog2e, g1.y * kLog2e, lane);
    const float e0 = __shfl_sync(~0u, sum.cum0, lane | 15), e1 = __shfl_sync(~0u, sum.cum1, lane | 15);
    Gates& o = gates[s];
    o.cum[lane] = sum.cum0, o.cum[lane + 32] = sum.cum1;
    o.d[lane] = g0.x, o.d[lane + 32] = g1.x;
    o.wd[lane] = g0.x * exp2_approx(e0 - sum.cum0), o.wd[lane + 32] = g1.x * exp2_approx(e1 - sum.cum1);
    o.wk[lane] = g0.x * exp2_approx(sum.rest0), o.wk[lane + 32] = g1.x * exp2_approx(sum.rest1);
    if (lane == 0) o.total = sum.total;
  };

  // The state: MT tiles of 16 rows by NT tiles of 8 columns per warp.
  constexpr int MTILES = KP / 16;
  constexpr int MT = MTILES >= 4 ? MTILES / 4 : 1;
  constexpr int NT = MTILES >= 4 ? VT / 8 : VT / 8 * MTILES / 4;
  const int m0 = MTILES >= 4 ? warp * MT : warp % MTILES;
  const int nt0 = MTILES >= 4 ? 0 : warp / MTILES * NT;
  float H[MT][NT][4];
  {
    const float* src = STATES_ONLY          ? nullptr
                       : cut.segments > 1   ? seg_state + ((size_t)pair * cut.segments + seg) * p.K * p.V
                       : p.H0               ? p.H0 + (size_t)pair * p.K * p.V
                                            : nullptr;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = (m0 + m) * 16 + g + (e >> 1) * 8, col = (nt0 + j) * 8 + c2 + (e & 1);
          H[m][j][e] = src && row < p.K && col < vw ? src[(size_t)row * p.V + v0 + col] : 0.f;
        }
  }
  // The state as the next chunk's bf16 operand and, where it is kept, as two bf16 values.
  auto put_state = [&](int chunk, int s) {
    uint16_t* kept = p.Hs ? p.Hs + ((size_t)pair * (chunks + 1) + chunk) * 2 * p.K * p.V : nullptr;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = (m0 + m) * 16 + g + r * 8, chunk16 = nt0 + j;
          const uint32_t hi = pack_bf16x2(H[m][j][2 * r], H[m][j][2 * r + 1]);
          st_shared_u32(Tile<VT>::at(tile_h(s), row, chunk16) + c2 * 2, hi);
          const int col = chunk16 * 8 + c2;
          if (kept && row < p.K && col < vw) {
            const uint32_t lo = pack_bf16x2(H[m][j][2 * r] - bf16_lo(hi), H[m][j][2 * r + 1] - bf16_hi(hi));
            uint16_t* at = kept + (size_t)row * p.V + v0 + col;
            const size_t plane = (size_t)p.K * p.V;
            if ((p.V & 1) == 0) {
              *reinterpret_cast<uint32_t*>(at) = hi;
              *reinterpret_cast<uint32_t*>(at + plane) = lo;
            } else {
              at[0] = (uint16_t)hi, at[plane] = (uint16_t)lo;
              if (col + 1 < vw) at[1] = (uint16_t)(hi >> 16), at[plane + 1] = (uint16_t)(lo >> 16);
            }
          }
        }
  };

  float decay = 0.f;  // log2 of the segment's decay
  if (first < last) {
    load_chunk(first, 0);
    if (rb == 0) put_gates(load_logits(first), 0);
  }
  if constexpr (!STATES_ONLY) put_state(first, 0);

  for (int chunk = first; chunk < last; ++chunk) {
    const int s = (chunk - first) & 1;
    cp_async_wait<0>();
    __syncthreads();
    const bool more = chunk + 1 < last;
    if (more) load_chunk(chunk + 1, s ^ 1);
    float2 logits = make_float2(0.f, 0.f);
    if (more && rb == 0) logits = load_logits(chunk + 1);
    const Gates& G = gates[s];

    // y of this warp's tokens, first from the state before the chunk.
    float y[8][4];
    uint32_t qa[KP / 16][4];
    float row_cum[2];
    if constexpr (!STATES_ONLY) {
      row_cum[0] = G.cum[rb * 16 + g];
      row_cum[1] = G.cum[rb * 16 + g + 8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[i][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < KP / 16; ++kk) {
        ldsm_x4(qa[kk], frag_at<KP>(tile_q(s), part_k_down, rb * 16, kk * 2));
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          uint32_t h[4];
          ldsm_x4_trans(h, frag_at<VT>(tile_h(s), part_v_down, kk * 16, np * 2));
          mma_bf16_16816(y[2 * np], qa[kk], h[0], h[1]);
          mma_bf16_16816(y[2 * np + 1], qa[kk], h[2], h[3]);
        }
      }
      const float e0 = exp2_approx(row_cum[0]), e1 = exp2_approx(row_cum[1]);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i][0] *= e0, y[i][1] *= e0, y[i][2] *= e1, y[i][3] *= e1;
    }
    const float whole = exp2_approx(G.total);
    if constexpr (STATES_ONLY) decay += G.total;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) H[m][j][e] *= whole;

#pragma unroll
    for (int j = 0; j < 4; ++j) {  // 16 tokens s at a time
      uint32_t vf[4][4];
#pragma unroll
      for (int np = 0; np < 4; ++np) ldsm_x4_trans(vf[np], frag_at<VT>(tile_v(s), part_v_down, j * 16, np * 2));
      if constexpr (!STATES_ONLY) {
        if (j <= rb) {
          float sc[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[i][e] = 0.f;
#pragma unroll
          for (int kk = 0; kk < KP / 16; ++kk) {
            uint32_t kf[4];
            ldsm_x4(kf, frag_at<KP>(tile_k(s), part_k_across, j * 16, kk * 2));
            mma_bf16_16816(sc[0], qa[kk], kf[0], kf[1]);
            mma_bf16_16816(sc[1], qa[kk], kf[2], kf[3]);
          }
          uint32_t pa[4];
          if (j < rb) {
            const float end = G.cum[j * 16 + 15];
            const float u0 = exp2_approx(row_cum[0] - end), u1 = exp2_approx(row_cum[1] - end);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float2 w = *reinterpret_cast<const float2*>(&G.wd[j * 16 + i * 8 + c2]);
              pa[2 * i] = pack_bf16x2(sc[i][0] * (u0 * w.x), sc[i][1] * (u0 * w.y));
              pa[2 * i + 1] = pack_bf16x2(sc[i][2] * (u1 * w.x), sc[i][3] * (u1 * w.y));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float2 cs = *reinterpret_cast<const float2*>(&G.cum[j * 16 + i * 8 + c2]);
              const float2 d = *reinterpret_cast<const float2*>(&G.d[j * 16 + i * 8 + c2]);
              float q[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int row = g + (e >> 1) * 8, col = i * 8 + c2 + (e & 1);
                const float m = exp2_approx(row_cum[e >> 1] - (e & 1 ? cs.y : cs.x)) * (e & 1 ? d.y : d.x);
                q[e] = col <= row ? sc[i][e] * m : 0.f;
              }
              pa[2 * i] = pack_bf16x2(q[0], q[1]);
              pa[2 * i + 1] = pack_bf16x2(q[2], q[3]);
            }
          }
#pragma unroll
          for (int np = 0; np < 4; ++np) {
            mma_bf16_16816(y[2 * np], pa, vf[np][0], vf[np][1]);
            mma_bf16_16816(y[2 * np + 1], pa, vf[np][2], vf[np][3]);
          }
        }
      }
      // The state's sum over these 16 tokens.
      const float2 w0 = *reinterpret_cast<const float2*>(&G.wk[j * 16 + c2]);
      const float2 w1 = *reinterpret_cast<const float2*>(&G.wk[j * 16 + 8 + c2]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint32_t kf[4], hi[4], lo[4];
        ldsm_x4_trans(kf, frag_at<KP>(tile_k(s), part_k_across, j * 16, (m0 + m) * 2));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float2 w = r < 2 ? w0 : w1;
          split_bf16x2(bf16_lo(kf[r]) * w.x, bf16_hi(kf[r]) * w.y, hi[r], lo[r]);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const int tile = MTILES >= 4 ? i : nt0 + i;
          // (a warp of a narrow state takes some of the column tiles: chosen without indexing)
          uint32_t b0 = vf[i >> 1][(i & 1) * 2], b1 = vf[i >> 1][(i & 1) * 2 + 1];
          if constexpr (MTILES < 4) {
#pragma unroll
            for (int o = 0; o < 8; ++o)
              if (o == tile) b0 = vf[o >> 1][(o & 1) * 2], b1 = vf[o >> 1][(o & 1) * 2 + 1];
          }
          mma_bf16_16816(H[m][i], hi, b0, b1);
          mma_bf16_16816(H[m][i], lo, b0, b1);
        }
      }
    }

    if constexpr (!STATES_ONLY) {
      // y += w_r v, out through shared memory (this warp's own rows of q, no longer needed).
      const uint32_t out = KP >= 64 ? tile_q(s) + rb * 16 * KP * 2 : base + 2 * S::kStage + 2 * S::kH + rb * 16 * VT * 2;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int col = i * 8 + c2;
        const float2 w = *reinterpret_cast<const float2*>(wr + col);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t v = ld_shared_u32(Tile<VT>::at(tile_v(s), rb * 16 + g + r * 8, i) + c2 * 2);
          st_shared_u32(Tile<VT>::at(out, g + r * 8, i) + c2 * 2,
                        pack_bf16x2(fmaf(w.x, bf16_lo(v), y[i][2 * r]), fmaf(w.y, bf16_hi(v), y[i][2 * r + 1])));
        }
      }
      __syncwarp();
      const long long t0 = (long long)chunk * L + rb * 16;
      uint16_t* yg = p.y + ((b * p.T + t0) * p.N + n) * p.V + v0;
      const long long ystride = (long long)p.N * p.V;
      if (vec) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = (lane >> 3) + i * 4, ch = lane & 7;
          if (t0 + row < p.T && ch * 8 < vw)
            *reinterpret_cast<uint4*>(yg + row * ystride + ch * 8) = ld_shared_v4(Tile<VT>::at(out, row, ch));
        }
      } else {
        for (int i = lane; i < 16 * VT; i += 32) {
          const int row = i / VT, col = i % VT;
          if (t0 + row < p.T && col < vw) {
            const uint32_t u = ld_shared_u32(Tile<VT>::at(out, row, col >> 3) + (col & 6) * 2);
            yg[row * ystride + col] = (uint16_t)(col & 1 ? u >> 16 : u);
          }
        }
      }
      if (more || (p.Hs && last == chunks)) put_state(chunk + 1, s ^ 1);
    }
    if (more && rb == 0) put_gates(logits, s ^ 1);
  }

  float* dst = STATES_ONLY ? seg_state + ((size_t)pair * cut.segments + seg) * p.K * p.V
               : seg == cut.segments - 1 && p.H_T ? p.H_T + (size_t)pair * p.K * p.V
                                                  : nullptr;
  if (STATES_ONLY && vt == 0 && tid == 0) seg_decay[pair * cut.segments + seg] = decay;
  if (!dst) return;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = (m0 + m) * 16 + g + (e >> 1) * 8, col = (nt0 + j) * 8 + c2 + (e & 1);
        if (row < p.K && col < vw) dst[(size_t)row * p.V + v0 + col] = H[m][j][e];
      }
}

// seg_state[seg] from the segment's own sum to the state before the segment, in place.
__global__ void __launch_bounds__(256)
    ssm_join_kernel(const float* __restrict__ H0, float* __restrict__ seg_state,
                    const float* __restrict__ seg_decay, int segments, int kv) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  const long long pair = blockIdx.y;
  if (i >= kv) return;
  float h = H0 ? H0[(size_t)pair * kv + i] : 0.f;
  float* s = seg_state + (size_t)pair * segments * kv + i;
  constexpr int kAhead = 8;  // segments loaded at once
  for (int j = 0; j < segments; j += kAhead) {
    float own[kAhead], decay[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (j + u + 1 < segments) {
        own[u] = s[(size_t)(j + u) * kv];
        decay[u] = seg_decay[pair * segments + j + u];
      }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (j + u < segments) s[(size_t)(j + u) * kv] = h;
      if (j + u + 1 < segments) h = fmaf(exp2_approx(decay[u]), h, own[u]);
    }
  }
}

int blocks_per_sm(int K) { return K <= 64 ? 3 : 2; }

// Segments so that at most two full waves of blocks run where the pairs alone are fewer than a
// wave; every segment of at least four chunks.
Cut cut_of(int B, int T, int N, int K, int V) {
  const long long units = (long long)B * N * ((V + VT - 1) / VT);
  const long long slots = 152LL * blocks_per_sm(K);
  const int chunks = ssm_chunks(T);
  Cut c{1, chunks > 0 ? chunks : 1};
  if (units >= slots || chunks < 8) return c;
  long long want = 2 * slots / units;
  if (want > chunks / 4) want = chunks / 4;
  if (want > 1024) want = 1024;
  if (want < 2) return c;
  c.per = (int)((chunks + want - 1) / want);
  c.segments = (chunks + c.per - 1) / c.per;
  return c;
}

template <int KP>
cudaError_t run(const SsmProblem& p, bool vec, cudaStream_t stream) {
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [] {
    attr = cudaFuncSetAttribute(ssm_chunk_kernel<KP, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Smem<KP, false>::kBytes);
    if (attr == cudaSuccess)
      attr = cudaFuncSetAttribute(ssm_chunk_kernel<KP, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  Smem<KP, true>::kBytes);
  });
  if (attr != cudaSuccess) return attr;
  const Cut cut = cut_of(p.B, p.T, p.N, p.K, p.V);
  const long long pairs = (long long)p.B * p.N;
  const unsigned units = (unsigned)(pairs * ((p.V + VT - 1) / VT));
  float* state = p.ws;
  float* decay = p.ws ? p.ws + (size_t)pairs * cut.segments * p.K * p.V : nullptr;
  if (cut.segments > 1) {
    ssm_chunk_kernel<KP, true><<<dim3(units, cut.segments - 1), kThreads, Smem<KP, true>::kBytes, stream>>>(
        p, cut, state, decay, vec);
    const int kv = p.K * p.V;
    ssm_join_kernel<<<dim3((kv + 255) / 256, (unsigned)pairs), 256, 0, stream>>>(p.H0, state, decay,
                                                                                 cut.segments, kv);
  }
  ssm_chunk_kernel<KP, false><<<dim3(units, cut.segments), kThreads, Smem<KP, false>::kBytes, stream>>>(
      p, cut, state, decay, vec);
  return cudaGetLastError();
}

bool rows16(const uint16_t* p, const Strides& s, int width) {
  return width % 8 == 0 && s.batch % 8 == 0 && s.token % 8 == 0 && aligned_to(p, 16);
}

}  // namespace

size_t ssm_forward_workspace_bytes(int B, int T, int N, int, int K, int V) {
  const Cut c = cut_of(B, T, N, K, V);
  return c.segments > 1 ? sizeof(float) * (size_t)B * N * c.segments * ((size_t)K * V + 1) : 0;
}

cudaError_t launch_ssm_forward(const SsmProblem& p, cudaStream_t stream) {
  const bool vec = rows16(p.q, p.sq, p.K) && rows16(p.k, p.sk, p.K) && rows16(p.v, p.sv, p.V) &&
                   aligned_to(p.y, 16);
  if (p.K <= 16) return run<16>(p, vec, stream);
  if (p.K <= 32) return run<32>(p, vec, stream);
  if (p.K <= 64) return run<64>(p, vec, stream);
  return run<128>(p, vec, stream);
}

}  // namespace m2rnn
