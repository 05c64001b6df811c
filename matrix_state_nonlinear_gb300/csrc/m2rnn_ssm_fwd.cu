// m2rnn_ssm_fwd.cu — the selective scan of a prompt in chunks of 128 tokens (see include/m2rnn.h).
//
// With c_t the sum of log f over a chunk up to token t, and H the state before the chunk,
//   y_t = exp(c_t) H^T q_t + sum_{s <= t} exp(c_t - c_s) d_s (q_t . k_s) v_s + w_r v_t
//   H  <- exp(c_127) H + sum_s k_s (exp(c_127 - c_s) d_s v_s)^T
// so that a chunk is four products on the 5th-generation tensor cores, a token per tensor-memory
// lane: S = q k^T, Y1 = q H, Y2 = P v (P = S decayed and masked), U = k^T (weighted v).
// One block walks the chunks of one (batch, head) pair and one tile of 64 value columns; eight
// warps do the element-wise work and a ninth issues the products and computes the gates.
//  * S is decayed in float32 and rounded to bf16 in tensor memory, the first operand of P v; H is
//    rounded to bf16 as an operand; y is bf16.  The state itself is float32 in registers and takes
//    U with float32 weights: the weighted v enters as two bf16 values (17 bits), two products.
//  * exp(c_t - c_s) is split at the end of s's block of 32, exp(c_t - c_end) exp(c_end - c_s), two
//    factors of at most one: one exponential per row and block instead of one per score.
//  * The next chunk's S and U are issued while this chunk's readout is being written, so that the
//    tensor cores' latency is off the chain: per chunk S -> P -> P v -> y and U -> H -> q H.
//  * Tiles are loaded by cp.async, one whole chunk ahead where shared memory allows (K <= 64).
// Where the pairs are fewer than the SMs, segments of a sequence run side by side
// (m2rnn_ssm_seg.cu).
#include <mutex>

#include "m2rnn_ssm_tc.cuh"

namespace m2rnn {
namespace {

constexpr int kCompute = 256;
constexpr int kThreads = kCompute + 32;
constexpr int L = kTokens;
constexpr int VT = kSsmColumns;

// Tensor memory columns.
constexpr int kColS = 0, kColP = 128, kColY1 = 192, kColY2 = 256, kColU = 320, kTmemCols = 512;

template <int KP>
struct Smem {
  static constexpr int kStages = KP <= 64 ? 3 : 2;
  static constexpr int kQ = L * KP * 2, kV = L * VT * 2;
  static constexpr int kStage = 2 * kQ + kV;
  static constexpr int kW = kStages * kStage;  // weighted v, high and low
  static constexpr int kH = kW + 2 * kV;
  static constexpr int kGates = kH + KP * VT * 2;
  static constexpr int kWr = kGates + 4 * (int)sizeof(ChunkGates);
  static constexpr int kBars = kWr + VT * 4;
  static constexpr int kBytes = kBars + 64 + 1024;  // and slack to align the tiles
  static_assert(kBytes <= 227 * 1024 && sizeof(ChunkGates) % 16 == 0, "");
};

template <int KP>
__global__ void __launch_bounds__(kThreads, 1)
    ssm_forward_kernel(SsmProblem p, SsmCut cut, int pieces, bool vec) {
  using S = Smem<KP>;
  constexpr int PANELS = KP / 64;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t base = smem_u32(smem);
  ChunkGates* gates = reinterpret_cast<ChunkGates*>(smem + S::kGates);
  float* wr = reinterpret_cast<float*>(smem + S::kWr);
  uint64_t* bar_s = reinterpret_cast<uint64_t*>(smem + S::kBars);  // S of the next chunk is done
  uint64_t* bar_q = bar_s + 1;  // q H
  uint64_t* bar_y = bar_s + 2;  // P v
  uint64_t* bar_u = bar_s + 3;  // U of the next chunk
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_s + 4);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) mbar_init(bar_s + i, 1);
    fence_mbar_init();
  }
  if (warp == 8) tmem_alloc(tmem_slot, kTmemCols);
  if (tid < VT) wr[tid] = tid < vw ? p.w_r[(size_t)n * p.V + v0 + tid] : 0.f;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto stage = [&](int i) { return base + i % S::kStages * S::kStage; };
  bool bad = false;

  if (warp == 8) {  // ------------------------------------------- products and gates
    const uint16_t* ag = p.a + b * p.sa.batch + n;
    const float alpha = p.alpha[n], beta = p.beta[n];
    auto put_gates = [&](int i) {
      if (i >= count) return;
      float a[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const long long t = (long long)(first + i) * L + 4 * lane + e;
        a[e] = t < p.T ? bf16_to_f(ag[t * p.sa.token]) : -INFINITY;
      }
      put_chunk_gates(gates[i & 3], a, alpha, beta, lane);
    };
    const uint32_t idesc_s = umma_idesc_bf16(128, 128, false);
    const uint32_t idesc_y = umma_idesc_bf16_ab(128, VT, false, true);
    const uint32_t idesc_u = umma_idesc_bf16_ab(KP, VT, true, true);
    const uint64_t dh = desc_mn(base + S::kH, KP), dw = desc_mn(base + S::kW, L);
    auto issue_s = [&](int i) {  // S = q k^T
      umma_loop<KP / 16, 2, 2, L * 8 - 8, L * 8 - 8>(tmem + kColS, desc_k(stage(i)), desc_k(stage(i) + S::kQ), idesc_s,
                                                     false);
      umma_commit(bar_s);
    };
    auto issue_u = [&](int i) {  // U = k^T (weighted v), high then low
      const uint64_t dk = desc_mn(stage(i) + S::kQ, L);
      umma_loop<L / 16, 128, 128>(tmem + kColU, dk, dw, idesc_u, false);
      umma_loop<L / 16, 128, 128>(tmem + kColU, dk, dw + (S::kV >> 4), idesc_u, true);
      umma_commit(bar_u);
    };
    put_gates(0);
    put_gates(1);
    __syncthreads();  // chunk 0, the first state and the first gates are in place
    fence_proxy_async_smem();
    if (lane == 0 && count > 0) issue_s(0);
    __syncwarp();
    __syncthreads();  // the first weighted v
    if (lane == 0 && count > 0) issue_u(0);
    __syncwarp();
    for (int i = 0; i < count; ++i) {
      if (sync_or(false)) break;  // P is written; chunk i + 1 is loaded
      tc_fence_after();
      if (lane == 0) {
        umma_loop<KP / 16, 2, 128, L * 8 - 8>(tmem + kColY1, desc_k(stage(i)), dh, idesc_y, false);
        umma_commit(bar_q);
        const uint64_t dv = desc_mn(stage(i) + 2 * S::kQ, L);
#pragma unroll
        for (int kk = 0; kk < L / 16; ++kk)
          umma_bf16_ta(tmem + kColY2, tmem + kColP + kk * 8, dv + kk * 128, idesc_y, kk > 0);
        umma_commit(bar_y);
        if (i + 1 < count) issue_s(i + 1);
      }
      __syncwarp();
      put_gates(i + 2);
      if (sync_or(false)) break;  // the next state and weighted v are written
      tc_fence_after();
      if (lane == 0 && i + 1 < count) issue_u(i + 1);
      __syncwarp();
    }
  } else {  // ------------------------------------------------------ element-wise
    const int quarter = warp & 3, half = warp >> 2;
    const int row = 32 * quarter + lane;  // token of the chunk, tensor-memory lane
    const uint32_t t_lane = tmem + ((uint32_t)(32 * quarter) << 16);
    TileLoader<64, L, kCompute> load_q[PANELS], load_k[PANELS];
    TileLoader<VT, L, kCompute> load_v;
#pragma unroll
    for (int x = 0; x < PANELS; ++x) {
      load_q[x].init(p.q + b * p.sq.batch + (long long)head * p.K + 64 * x, p.sq.token, p.K - 64 * x, tid);
      load_k[x].init(p.k + b * p.sk.batch + (long long)head * p.K + 64 * x, p.sk.token, p.K - 64 * x, tid);
    }
    load_v.init(p.v + b * p.sv.batch + (long long)n * p.V + v0, p.sv.token, vw, tid);
    auto load = [&](int i) {
      if (i < count) {
        const long long t0 = (long long)(first + i) * L;
        const int rows = (int)min((long long)L, p.T - t0);
#pragma unroll
        for (int x = 0; x < PANELS; ++x) {
          load_q[x].load(stage(i) + panel(x, L), t0, rows, vec, tid);
          load_k[x].load(stage(i) + S::kQ + panel(x, L), t0, rows, vec, tid);
        }
        load_v.load(stage(i) + 2 * S::kQ, t0, rows, vec, tid);
      }
      cp_async_commit();
    };
    load(0);
    load(1);

    // The state: this thread's row of K and 32 of the 64 columns.  With K <= 64 the product has 64
    // rows, 16 in each quarter's first lanes.
    const int hrow = KP > 64 ? row : 16 * quarter + lane;
    const bool has_row = (KP > 64 || lane < 16) && hrow < p.K;
    const int hcol = 32 * half;
    float H[32];
    const float* src = cut.segments > 1 ? p.ws + ((size_t)pair * pieces + seg * cut.fine) * plane
                       : p.H0           ? p.H0 + pair * plane
                                        : nullptr;
#pragma unroll
    for (int c = 0; c < 32; ++c)
      H[c] = src && has_row && hcol + c < vw ? src[(size_t)hrow * p.V + v0 + hcol + c] : 0.f;
    uint16_t* kept = p.Hs ? p.Hs + (size_t)pair * (chunks + 1) * 2 * plane + (size_t)hrow * p.V + v0 + hcol : nullptr;
    // The state before chunk i as the bf16 operand and, where it is kept, as two bf16 values.
    auto put_state = [&](int i, bool keep) {
      if (KP <= 64 && lane >= 16) return;
      uint16_t* to = kept + (size_t)(first + i) * 2 * plane;
      keep = keep && kept && has_row;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_bf16x2(make_float2(H[8 * c + 2 * e], H[8 * c + 2 * e + 1]), hi[e], lo[e]);
        st_shared_v4(Tile<VT>::at(base + S::kH, hrow, hcol / 8 + c), make_uint4(hi[0], hi[1], hi[2], hi[3]));
        if (!keep) continue;
        if (vec) {
          if (hcol + 8 * c < vw) {
            *reinterpret_cast<uint4*>(to + 8 * c) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(to + plane + 8 * c) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (hcol + 8 * c + e < vw) {
              to[8 * c + e] = (uint16_t)(hi[e >> 1] >> (16 * (e & 1)));
              to[plane + 8 * c + e] = (uint16_t)(lo[e >> 1] >> (16 * (e & 1)));
            }
        }
      }
    };
    // Half a token's v of chunk i, weighted, as two bf16 values.
    auto put_weighted = [&](int i) {
      const float w = gates[i & 3].wk[row];
      const float2 w2 = make_float2(w, w);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t at = Tile<VT>::at(0, row, 4 * half + c);
        float2 f[4];
        uint32_t hi[4], lo[4];
        unpack8(ld_shared_v4(stage(i) + 2 * S::kQ + at), f);
#pragma unroll
        for (int e = 0; e < 4; ++e) split_bf16x2(mul2(f[e], w2), hi[e], lo[e]);
        st_shared_v4(base + S::kW + at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
        st_shared_v4(base + S::kW + S::kV + at, make_uint4(lo[0], lo[1], lo[2], lo[3]));
      }
    };
    put_state(0, true);
    cp_async_wait<1>();
    fence_proxy_async_smem();
    __syncthreads();
    if (count > 0) put_weighted(0);
    fence_proxy_async_smem();
    __syncthreads();

    auto wait = [&](uint64_t* bar, uint32_t parity) {
      bad |= !mbar_wait_bounded(bar, parity, kWaitLimitCycles);
      __syncwarp();
      tc_fence_after();
    };
    bool stop = false;
    for (int i = 0; i < count; ++i) {
      const ChunkGates& G = gates[i & 3];
      const uint32_t parity = i & 1;
      const float cum = G.cum[row];
      // P from S: block cb of 32 columns against the quarter's own block of 32 rows.
      wait(bar_s, parity);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int cb = 2 * half + x;
        uint32_t out[16];
        if (cb > quarter) {
#pragma unroll
          for (int e = 0; e < 16; ++e) out[e] = 0u;
        } else {
          float s[32];
          tmem_ld32(t_lane + kColS + 32 * cb, s);
          tmem_wait_ld();
          if (cb < quarter) {
            const float u = exp2_approx(cum - G.cum[32 * cb + 31]);
            const float2 u2 = make_float2(u, u);
            const float4* w = reinterpret_cast<const float4*>(G.wd + 32 * cb);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 wv = w[e];
              const float2 a = mul2(make_float2(s[4 * e], s[4 * e + 1]), mul2(u2, make_float2(wv.x, wv.y)));
              const float2 c = mul2(make_float2(s[4 * e + 2], s[4 * e + 3]), mul2(u2, make_float2(wv.z, wv.w)));
              out[2 * e] = pack_bf16x2(a.x, a.y);
              out[2 * e + 1] = pack_bf16x2(c.x, c.y);
            }
          } else {
            const float4* w = reinterpret_cast<const float4*>(G.diag + 32 * cb);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 wv = w[e];
              const float m[4] = {exp2_approx(cum - wv.x), exp2_approx(cum - wv.y), exp2_approx(cum - wv.z),
                                  exp2_approx(cum - wv.w)};
              float q[4];
#pragma unroll
              for (int z = 0; z < 4; ++z) q[z] = 4 * e + z <= lane ? s[4 * e + z] * m[z] : 0.f;
              out[2 * e] = pack_bf16x2(q[0], q[1]);
              out[2 * e + 1] = pack_bf16x2(q[2], q[3]);
            }
          }
        }
        tmem_st16(t_lane + kColP + 16 * cb, out);
      }
      tmem_wait_st();
      cp_async_wait<0>();
      fence_proxy_async_smem();
      tc_fence_before();
      if (stop = sync_or(bad)) break;
      if constexpr (S::kStages > 2) load(i + 2);

      // The state after the chunk; H's tile is free once q H is done.
      wait(bar_u, parity);
      {
        float u[32];
        tmem_ld32(t_lane + kColU + hcol, u);
        const float e = exp2_approx(G.total);
        const float2 e2 = make_float2(e, e);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const float2 h = fma2(e2, make_float2(H[c], H[c + 1]), make_float2(u[c], u[c + 1]));
          H[c] = h.x, H[c + 1] = h.y;
        }
      }
      wait(bar_q, parity);
      put_state(i + 1, i + 1 < count || first + count == chunks);
      if (i + 1 < count) put_weighted(i + 1);
      fence_proxy_async_smem();
      tc_fence_before();
      if (stop = sync_or(bad)) break;

      // y: half a token's 64 columns, out through shared memory (this half row of q, done with).
      wait(bar_y, parity);
      {
        float y1[32], y2[32];
        tmem_ld32(t_lane + kColY1 + hcol, y1);
        tmem_ld32(t_lane + kColY2 + hcol, y2);
        const float e = exp2_approx(cum);
        const float2 e2 = make_float2(e, e);
        tmem_wait_ld();
        const uint32_t tq = stage(i), tv = stage(i) + 2 * S::kQ;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t at = Tile<VT>::at(0, row, 4 * half + c);
          float2 v[4];
          uint32_t o[4];
          unpack8(ld_shared_v4(tv + at), v);
          const float4 w0 = *reinterpret_cast<const float4*>(wr + hcol + 8 * c);
          const float4 w1 = *reinterpret_cast<const float4*>(wr + hcol + 8 * c + 4);
          const float2 w[4] = {make_float2(w0.x, w0.y), make_float2(w0.z, w0.w), make_float2(w1.x, w1.y),
                               make_float2(w1.z, w1.w)};
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const int k = 8 * c + 2 * z;
            const float2 r = fma2(w[z], v[z], fma2(e2, make_float2(y1[k], y1[k + 1]), make_float2(y2[k], y2[k + 1])));
            o[z] = pack_bf16x2(r.x, r.y);
          }
          st_shared_v4(tq + at, make_uint4(o[0], o[1], o[2], o[3]));
        }
        __syncwarp();
        const long long t0 = (long long)(first + i) * L + 32 * quarter;
        uint16_t* yg = p.y + ((b * p.T + t0) * p.N + n) * p.V + v0 + hcol;
        const long long ystride = (long long)p.N * p.V;
        if (vec) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int r = (lane >> 2) + 8 * x, ch = lane & 3;
            if (t0 + r < p.T && hcol + ch * 8 < vw)
              *reinterpret_cast<uint4*>(yg + r * ystride + ch * 8) =
                  ld_shared_v4(Tile<VT>::at(tq, 32 * quarter + r, 4 * half + ch));
          }
        } else {
          for (int x = lane; x < 32 * 32; x += 32) {
            const int r = x >> 5, col = x & 31;
            if (t0 + r < p.T && hcol + col < vw) {
              const uint32_t u =
                  ld_shared_u32(Tile<VT>::at(tq, 32 * quarter + r, 4 * half + (col >> 3)) + (col & 6) * 2);
              yg[r * ystride + col] = (uint16_t)(col & 1 ? u >> 16 : u);
            }
          }
        }
      }
      if constexpr (S::kStages == 2) {
        named_bar_sync(1, kCompute);  // every warp is done with the chunk's tiles
        load(i + 2);
      }
    }
    if (stop && tid == 0) atomicExch(p.status, kStatusTimeout);
    cp_async_wait<0>();
    if (!stop && p.H_T && first + count == chunks && has_row) {
      float* dst = p.H_T + pair * plane + (size_t)hrow * p.V + v0 + hcol;
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (hcol + c < vw) dst[c] = H[c];
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, kTmemCols);
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
  return p.K <= 64 ? run<64>(p, cut, vec, stream) : run<128>(p, cut, vec, stream);
}

}  // namespace m2rnn
