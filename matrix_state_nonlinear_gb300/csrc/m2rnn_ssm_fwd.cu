// m2rnn_ssm_fwd.cu — the selective scan of a prompt in chunks of 64 tokens (see include/m2rnn.h).
//
// With c_t the sum of log f over a chunk up to token t, and H the state before the chunk,
//   y_t = exp(c_t) H^T q_t + sum_{s <= t} exp(c_t - c_s) d_s (q_t . k_s) v_s + w_r v_t
//   H  <- exp(c_63) H + sum_s (exp(c_63 - c_s) d_s k_s) v_s^T
// so that a chunk is five matrix products.  One block of twelve warps walks the chunks of one
// (batch, head) pair and one tile of 64 value columns, in step, one chunk per step:
//  * four warps carry the state, K / 4 rows each in float32 registers, and leave it as bf16 in
//    shared memory for the next step;
//  * two sets of four warps compute y, each set every other chunk over two steps (16 tokens a
//    warp): the product with the state before the chunk in its first step, which is the only step
//    that reads that state, the scores and their product with v over both.
// The state's chain, the only serial part, is then a third of the work, and an SM's four quarters
// hold three warps each of equal work (the two sets deal the triangle's rows in opposite orders).
//  * Scores above the diagonal's 16 x 16 block are not computed.  Scores are decayed in float32 and
//    rounded to bf16 as the operand of the product with v; the state is rounded to bf16 as the
//    operand of H^T q; y is bf16.  The state's own update keeps the float32 weights: weight times k
//    enters as two bf16 values (17 bits), two products.
//  * exp(c_t - c_s) is split at the end of s's block of 16, exp(c_t - c_end) exp(c_end - c_s), two
//    factors of at most one: one exponential per row and block instead of one per score.
//  * Tiles of q, k and v are loaded by cp.async one or two steps ahead.
// Where the pairs are fewer than the SMs, segments of a sequence run side by side
// (m2rnn_ssm_seg.cu).
#include <mutex>

#include "m2rnn_ssm_mma.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 384;
constexpr int L = kSsmChunk;
constexpr int VT = kSsmColumns;

struct alignas(16) Gates {  // of one chunk, per token; read in pairs
  float cum[L];   // log2 of the decay from the chunk's start, the token's own included
  float d[L];     // step size
  float wd[L];    // d times the decay from the token to the end of its 16
  float wk[L];    // d times the decay from the token to the chunk's end
  float total;    // log2 of the whole chunk's decay
};

template <int KP>
struct Smem {
  static constexpr int kStages = KP <= 64 ? 4 : 3;  // a chunk's tiles live for two steps
  static constexpr int kQ = L * KP * 2, kV = L * VT * 2;
  static constexpr int kStage = 2 * kQ + kV;
  static constexpr int kPlane = KP * VT * 2;  // the state as bf16, and the remainder's plane
  static constexpr int kH = kStages * kStage;
  static constexpr int kY = kH + 4 * kPlane;  // y on its way out: q's rows where they are wide enough
  static constexpr int kGates = kY + (KP >= 64 ? 0 : 8 * 16 * VT * 2);
  static constexpr int kWr = kGates + 8 * (int)sizeof(Gates);
  static constexpr int kBytes = kWr + VT * 4;
  static_assert(kGates % 16 == 0 && sizeof(Gates) % 16 == 0 && kBytes <= 227 * 1024, "");
};

template <int KP>
__global__ void __launch_bounds__(kThreads, 1)
    ssm_forward_kernel(SsmProblem p, SsmCut cut, int pieces, bool vec) {
  using S = Smem<KP>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = smem_u32(smem);
  Gates* gates = reinterpret_cast<Gates*>(smem + S::kGates);
  float* wr = reinterpret_cast<float*>(smem + S::kWr);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int set = warp >> 2, w4 = warp & 3;  // set 0: the state; 1, 2: y of even and odd chunks
  const int g = lane >> 2, c2 = (lane & 3) * 2;
  const int vtiles = (p.V + VT - 1) / VT;
  const int vt = blockIdx.x % vtiles, seg = blockIdx.y;
  const long long pair = blockIdx.x / vtiles;
  const int n = (int)(pair % p.N);
  const long long b = pair / p.N;
  const int head = (int)((long long)n * p.Nqk / p.N);
  const int chunks = ssm_chunks(p.T);
  const int first = seg * cut.per, count = min(chunks, first + cut.per) - first;
  const int v0 = vt * VT, vw = min(VT, p.V - v0);
  const size_t plane = (size_t)p.K * p.V;
  uint16_t* kept = p.Hs ? p.Hs + (size_t)pair * (chunks + 1) * 2 * plane + v0 : nullptr;

  const uint16_t* ag = p.a + b * p.sa.batch + n;
  const float alpha = p.alpha[n], beta = p.beta[n];
  TileLoader<KP, L, kThreads> load_q, load_k;
  TileLoader<VT, L, kThreads> load_v;
  load_q.init(p.q + b * p.sq.batch + (long long)head * p.K, p.sq.token, p.K, tid);
  load_k.init(p.k + b * p.sk.batch + (long long)head * p.K, p.sk.token, p.K, tid);
  load_v.init(p.v + b * p.sv.batch + (long long)n * p.V + v0, p.sv.token, vw, tid);
  auto stage = [&](int i) { return base + i % S::kStages * S::kStage; };
  auto load = [&](int i) {
    if (i < count) {
      const long long t0 = (long long)(first + i) * L;
      const int rows = min(L, p.T - (first + i) * L);
      load_q.load(stage(i), t0, rows, vec, tid);
      load_k.load(stage(i) + S::kQ, t0, rows, vec, tid);
      load_v.load(stage(i) + 2 * S::kQ, t0, rows, vec, tid);
    }
    cp_async_commit();
  };
  // One warp's chunk: tokens lane and lane + 32.
  auto put_gates = [&](int i) {
    if (i >= count) return;
    const int t = (first + i) * L + lane;
    const float2 g0 = ssm_gate(t < p.T ? bf16_to_f(ag[t * p.sa.token]) : -INFINITY, alpha, beta);
    const float2 g1 = ssm_gate(t + 32 < p.T ? bf16_to_f(ag[(t + 32) * p.sa.token]) : -INFINITY, alpha, beta);
    const ChunkSums sum = chunk_sums(g0.y * kLog2e, g1.y * kLog2e, lane);
    const float e0 = __shfl_sync(~0u, sum.cum0, lane | 15), e1 = __shfl_sync(~0u, sum.cum1, lane | 15);
    Gates& o = gates[i & 7];
    o.cum[lane] = sum.cum0, o.cum[lane + 32] = sum.cum1;
    o.d[lane] = g0.x, o.d[lane + 32] = g1.x;
    o.wd[lane] = g0.x * exp2_approx(e0 - sum.cum0), o.wd[lane + 32] = g1.x * exp2_approx(e1 - sum.cum1);
    o.wk[lane] = g0.x * exp2_approx(sum.rest0), o.wk[lane + 32] = g1.x * exp2_approx(sum.rest1);
    if (lane == 0) o.total = sum.total;
  };
  if (tid < VT) wr[tid] = tid < vw ? p.w_r[(size_t)n * p.V + v0 + tid] : 0.f;
  load(0);
  if constexpr (S::kStages == 4) load(1);
  const uint32_t part_k_down = lane_part<KP>(lane, true), part_k_across = lane_part<KP>(lane, false);
  const uint32_t part_v_down = lane_part<VT>(lane, true);
  // Every set waits, joins the block and starts the next load in the same places.
  auto step = [&](int i) {
    if constexpr (S::kStages == 4)
      cp_async_wait<1>();
    else
      cp_async_wait<0>();
    __syncthreads();
    load(i + S::kStages - 2);
  };

  if (set == 0) {  // ---------------------------------------------------- the state
    using T = StateTiles<KP, VT>;
    const int m0 = T::row_tile(w4), nt0 = T::col_tile(w4);
    float H[T::MT][T::NT][4];
    const float* src = cut.segments > 1 ? p.ws + ((size_t)pair * pieces + seg * cut.fine) * plane
                       : p.H0           ? p.H0 + pair * plane
                                        : nullptr;
    auto at = [&](int m, int j, int e) {
      return (size_t)((m0 + m) * 16 + g + (e >> 1) * 8) * p.V + v0 + (nt0 + j) * 8 + c2 + (e & 1);
    };
    auto in = [&](int m, int j, int e) {
      return (m0 + m) * 16 + g + (e >> 1) * 8 < p.K && (nt0 + j) * 8 + c2 + (e & 1) < vw;
    };
#pragma unroll
    for (int m = 0; m < T::MT; ++m)
#pragma unroll
      for (int j = 0; j < T::NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) H[m][j][e] = src && in(m, j, e) ? src[at(m, j, e)] : 0.f;
    // The state before chunk i as bf16, with the remainder where states are kept.
    auto put_state = [&](int i) {
      const uint32_t to = base + S::kH + (i & 1) * 2 * S::kPlane;
#pragma unroll
      for (int m = 0; m < T::MT; ++m)
#pragma unroll
        for (int j = 0; j < T::NT; ++j)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t a = Tile<VT>::at(to, (m0 + m) * 16 + g + r * 8, nt0 + j) + c2 * 2;
            const float2 h = make_float2(H[m][j][2 * r], H[m][j][2 * r + 1]);
            const uint32_t hi = pack_bf16x2(h.x, h.y);
            st_shared_u32(a, hi);
            if (kept) {
              const float2 rest = sub2(h, bf16x2_to_float2(hi));
              st_shared_u32(a + S::kPlane, pack_bf16x2(rest.x, rest.y));
            }
          }
    };
    put_state(0);
    put_gates(w4);
    for (int i = 0; i < count; ++i) {
      step(i);
      const Gates& G = gates[i & 7];
      const uint32_t tk = stage(i) + S::kQ, tv = stage(i) + 2 * S::kQ;
      scale_state<T>(H, exp2_approx(G.total));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t vf[4][4];
#pragma unroll
        for (int np = 0; np < 4; ++np) ldsm_x4_trans(vf[np], frag_at<VT>(tv, part_v_down, j * 16, np * 2));
        add_outer<KP, T>(H, tk, part_k_across, G.wk, vf, j, m0, nt0, c2);
      }
      put_state(i + 1);
    }
    step(count);
    if (p.H_T && first + count == chunks) {
#pragma unroll
      for (int m = 0; m < T::MT; ++m)
#pragma unroll
        for (int j = 0; j < T::NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (in(m, j, e)) p.H_T[pair * plane + at(m, j, e)] = H[m][j][e];
    }
  } else {  // ------------------------------------------------------------ y
    const int rb = set == 1 ? w4 : 3 - w4;  // this warp's 16 tokens of a chunk
    const int odd = set - 1;
    float y[8][4];
    uint32_t qa[KP <= 64 ? KP / 16 : 1][4];  // q of those tokens, kept where registers allow
    float row_cum[2] = {0.f, 0.f};
    // The scores of tokens rb against block j, decayed, times v.
    auto add_block = [&](const Gates& G, uint32_t tile, int j) {
      float sc[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[i][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < KP / 16; ++kk) {
        uint32_t kf[4], qr[4];
        ldsm_x4(kf, frag_at<KP>(tile + S::kQ, part_k_across, j * 16, kk * 2));
        if constexpr (KP > 64) {
          ldsm_x4(qr, frag_at<KP>(tile, part_k_down, rb * 16, kk * 2));
          mma_bf16_16816(sc[0], qr, kf[0], kf[1]);
          mma_bf16_16816(sc[1], qr, kf[2], kf[3]);
        } else {
          mma_bf16_16816(sc[0], qa[kk], kf[0], kf[1]);
          mma_bf16_16816(sc[1], qa[kk], kf[2], kf[3]);
        }
      }
      uint32_t pa[4];
      if (j < rb) {
        const float end = G.cum[j * 16 + 15];
        const float u0 = exp2_approx(row_cum[0] - end), u1 = exp2_approx(row_cum[1] - end);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 w = *reinterpret_cast<const float2*>(&G.wd[j * 16 + i * 8 + c2]);
          const float2 s0 = mul2(make_float2(sc[i][0], sc[i][1]), mul2(w, make_float2(u0, u0)));
          const float2 s1 = mul2(make_float2(sc[i][2], sc[i][3]), mul2(w, make_float2(u1, u1)));
          pa[2 * i] = pack_bf16x2(s0.x, s0.y);
          pa[2 * i + 1] = pack_bf16x2(s1.x, s1.y);
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
        uint32_t vf[4];
        ldsm_x4_trans(vf, frag_at<VT>(tile + 2 * S::kQ, part_v_down, j * 16, np * 2));
        mma_bf16_16816(y[2 * np], pa, vf[0], vf[1]);
        mma_bf16_16816(y[2 * np + 1], pa, vf[2], vf[3]);
      }
    };
    const int early = rb == 3 ? 1 : 0;  // blocks of scores in the first step
    for (int i = 0; i <= count; ++i) {
      step(i);
      if ((i & 1) == odd) {
        // First step of chunk i: from the state before it.
        if (i < count) {
          const Gates& G = gates[i & 7];
          row_cum[0] = G.cum[rb * 16 + g];
          row_cum[1] = G.cum[rb * 16 + g + 8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[j][e] = 0.f;
          const uint32_t th = base + S::kH + (i & 1) * 2 * S::kPlane;
#pragma unroll
          for (int kk = 0; kk < KP / 16; ++kk) {
            uint32_t (&qr)[4] = qa[KP <= 64 ? kk : 0];
            ldsm_x4(qr, frag_at<KP>(stage(i), part_k_down, rb * 16, kk * 2));
#pragma unroll
            for (int np = 0; np < 4; ++np) {
              uint32_t h[4];
              ldsm_x4_trans(h, frag_at<VT>(th, part_v_down, kk * 16, np * 2));
              mma_bf16_16816(y[2 * np], qr, h[0], h[1]);
              mma_bf16_16816(y[2 * np + 1], qr, h[2], h[3]);
            }
          }
          const float e0 = exp2_approx(row_cum[0]), e1 = exp2_approx(row_cum[1]);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 a = mul2(make_float2(y[j][0], y[j][1]), make_float2(e0, e0));
            const float2 c = mul2(make_float2(y[j][2], y[j][3]), make_float2(e1, e1));
            y[j][0] = a.x, y[j][1] = a.y, y[j][2] = c.x, y[j][3] = c.y;
          }
          if (early) add_block(G, stage(i), 0);
        }
        if ((i & 6) == (odd ? 6 : 2)) put_gates((i & ~3) + 4 + w4);  // the next four chunks', one per warp
      } else {
        // The state before chunk i on its way to memory.
        if (kept && (i < count || first + count == chunks)) {
          const uint32_t th = base + S::kH + (i & 1) * 2 * S::kPlane;
          uint16_t* to = kept + (size_t)(first + i) * 2 * plane;
          if (vec) {
            constexpr int kPieces = KP * (VT / 8) / 128;
#pragma unroll
            for (int x = 0; x < kPieces; ++x) {
              const int id = (w4 * 32 + lane) + x * 128, row = id / (VT / 8), ch = id % (VT / 8);
              if (row < p.K && ch * 8 < vw) {
                uint16_t* o = to + (size_t)row * p.V + ch * 8;
                *reinterpret_cast<uint4*>(o) = ld_shared_v4(Tile<VT>::at(th, row, ch));
                *reinterpret_cast<uint4*>(o + plane) = ld_shared_v4(Tile<VT>::at(th + S::kPlane, row, ch));
              }
            }
          } else {
            for (int id = w4 * 32 + lane; id < KP * VT; id += 128) {
              const int row = id / VT, col = id % VT;
              if (row < p.K && col < vw) {
                const uint32_t a = Tile<VT>::at(th, row, col >> 3) + (col & 6) * 2;
                const uint32_t hi = ld_shared_u32(a), lo = ld_shared_u32(a + S::kPlane);
                to[(size_t)row * p.V + col] = (uint16_t)(col & 1 ? hi >> 16 : hi);
                to[(size_t)row * p.V + col + plane] = (uint16_t)(col & 1 ? lo >> 16 : lo);
              }
            }
          }
        }
        // Second step of chunk i - 1.
        if (i > 0) {
          const int c = i - 1;
          const Gates& G = gates[c & 7];
          const uint32_t tile = stage(c), tv = tile + 2 * S::kQ;
          for (int j = early; j <= rb; ++j) add_block(G, tile, j);
          // y += w_r v, out through shared memory (this warp's own rows of q, no longer needed).
          const uint32_t out = KP >= 64 ? tile + rb * 16 * KP * 2 : base + S::kY + (warp - 4) * 16 * VT * 2;
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 w = *reinterpret_cast<const float2*>(wr + j * 8 + c2);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t v = ld_shared_u32(Tile<VT>::at(tv, rb * 16 + g + r * 8, j) + c2 * 2);
              const float2 o = fma2(w, bf16x2_to_float2(v), make_float2(y[j][2 * r], y[j][2 * r + 1]));
              st_shared_u32(Tile<VT>::at(out, g + r * 8, j) + c2 * 2, pack_bf16x2(o.x, o.y));
            }
          }
          __syncwarp();
          const long long t0 = (long long)(first + c) * L + rb * 16;
          uint16_t* yg = p.y + ((b * p.T + t0) * p.N + n) * p.V + v0;
          const long long ystride = (long long)p.N * p.V;
          if (vec) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int row = (lane >> 3) + x * 4, ch = lane & 7;
              if (t0 + row < p.T && ch * 8 < vw)
                *reinterpret_cast<uint4*>(yg + row * ystride + ch * 8) = ld_shared_v4(Tile<VT>::at(out, row, ch));
            }
          } else {
            for (int x = lane; x < 16 * VT; x += 32) {
              const int row = x / VT, col = x % VT;
              if (t0 + row < p.T && col < vw) {
                const uint32_t u = ld_shared_u32(Tile<VT>::at(out, row, col >> 3) + (col & 6) * 2);
                yg[row * ystride + col] = (uint16_t)(col & 1 ? u >> 16 : u);
              }
            }
          }
        }
      }
    }
  }
  cp_async_wait<0>();
}

template <int KP>
cudaError_t run(const SsmProblem& p, const SsmCut& cut, bool vec, cudaStream_t stream) {
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [] {
    attr = cudaFuncSetAttribute(ssm_forward_kernel<KP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Smem<KP>::kBytes);
  });
  if (attr != cudaSuccess) return attr;
  const unsigned units = (unsigned)((long long)p.B * p.N * ((p.V + VT - 1) / VT));
  ssm_forward_kernel<KP><<<dim3(units, cut.segments), kThreads, Smem<KP>::kBytes, stream>>>(
      p, cut, ssm_pieces(cut, p.T), vec);
  return cudaGetLastError();
}

}  // namespace

size_t ssm_forward_workspace_bytes(int B, int T, int N, int, int K, int V) {
  return sizeof(float) * ssm_segment_floats(ssm_cut(B, T, N, V), B, T, N, K, V);
}

cudaError_t launch_ssm_forward(const SsmProblem& p, cudaStream_t stream) {
  const bool vec = rows_of_16(p.q, p.sq, p.K) && rows_of_16(p.k, p.sk, p.K) && rows_of_16(p.v, p.sv, p.V) &&
                   aligned_to(p.y, 16);
  const SsmCut cut = ssm_cut(p.B, p.T, p.N, p.V);
  if (cut.segments > 1) {
    SegmentProblem s{p.k, p.v, p.a, p.alpha, p.beta, p.H0, p.sk, p.sv, p.sa, p.B, p.T, p.N, p.Nqk, p.K, p.V, p.ws};
    const cudaError_t err = launch_ssm_segments(s, cut, false, vec, stream);
    if (err != cudaSuccess) return err;
  }
  if (p.K <= 16) return run<16>(p, cut, vec, stream);
  if (p.K <= 32) return run<32>(p, cut, vec, stream);
  if (p.K <= 64) return run<64>(p, cut, vec, stream);
  return run<128>(p, cut, vec, stream);
}

}  // namespace m2rnn
