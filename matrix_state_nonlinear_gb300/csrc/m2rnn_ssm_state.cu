// m2rnn_ssm_state.cu — the scan's states alone: from tokens to the state, forwards, or to the
// state's gradient, backwards.
//
//   forwards:   H <- exp(c_127) H + sum_s k_s (exp(c_127 - c_s) d_s v_s)^T      (reads k, v)
//   backwards:  G <- exp(c_127) G + sum_t q_t (exp(c_t) dy_t)^T                 (reads q, dy)
// over chunks of 128 tokens (c: sum of log f over the chunk).  Two uses:
//  * pieces: where there are fewer (batch, head) pairs than SMs, a pair's sequence is cut into
//    pieces, each piece's own state from zero found side by side, and a second launch chains them
//    into the state before (after) each; the main kernels start there;
//  * a training step's states: H before every chunk for the backward; and the backward's first
//    pass, G after every chunk, with <G, H>, H the state before the chunk: what reaches across it.
//    Kept as two bf16 values each, through shared memory so that whole rows leave at once.
// Products on the 5th-generation tensor cores: one of 128 x 16 steps per chunk, the weighted y in
// two bf16 values (17 bits) side by side as its second operand; warps by role as in the forward kernel.
// Measured: 87 us for the pieces of 65536 tokens of 16 heads, K = 64, V = 128 (weighing y in its eight warps
// bounds it; sixteen, at 72 registers, took as long and the kept states longer); kept states of 4 x 8192
// tokens of 32 heads, K = 128, V = 64: H 85 us (0.4 GB, 4.7 TB/s), G with <G, H> 136 us (0.67 GB,
// 4.9 TB/s), near the memory's rate.
#include "m2rnn_ssm_tc.cuh"

namespace m2rnn {
namespace {

constexpr int L = kTokens;
constexpr int VT = kSsmColumns;
constexpr int kWarpState = 8, kWarpMma = 16, kWarpLoad = 17, kWarpGate = 18, kWarps = 20;  // 0..7: weights
constexpr int kThreads = 32 * kWarps;
constexpr int kTmemCols = 256;  // two products

struct alignas(16) Weights {
  float w[L];
  float l[L];   // scratch of the gates
  float total;  // log2 of the chunk's decay
};

template <int KP, bool REVERSE, bool KEEP>
struct Smem {
  static constexpr int kStages = KEEP && KP > 64 ? 2 : 3;
  // Weighted y of two chunks, so that weighing and the product overlap: 142 -> 112 us for three pieces of
  // 65536 tokens of 16 heads, K = 64, V = 128.  (Backwards with K = 128 there is no room beside H; the
  // traffic of the states bounds that one.)
  static constexpr int kW2 = KEEP && REVERSE && KP > 64 ? 1 : 2;
  static constexpr int kX = L * KP * 2, kY = L * VT * 2;
  static constexpr int kStage = kX + kY;
  static constexpr int kW = kStages * kStage;  // weighted y, high and low
  static constexpr int kKept = kW + kW2 * 2 * kY;  // a state on its way out, high and low; and H on its way in
  static constexpr int kHs = kKept + (KEEP ? 2 * KP * VT * 2 : 0);
  static constexpr int kWeights = kHs + (KEEP && REVERSE ? 2 * KP * VT * 2 : 0);
  static constexpr int kBars = kWeights + 4 * (int)sizeof(Weights);
  static constexpr int kBytes = kBars + 256 + 1024;
  static_assert(kBytes <= 227 * 1024, "");
};

struct Bars {
  uint64_t full[3], empty[3];
  uint64_t gate[4], gate_free[4];
  uint64_t u[2], u_free[2], w[2];  // U done, read; weighted y written
  uint64_t put, put_free, hs, hs_free;  // kept state written, on its way; H loaded, read
  uint32_t tmem;
  int abort;
};

template <int KP, bool REVERSE, bool KEEP>
__global__ void __launch_bounds__(kThreads, 1)
    ssm_state_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_y,
                     const __grid_constant__ CUtensorMap map_kept, const __grid_constant__ CUtensorMap map_hs,
                     StateProblem p, bool tma) {
  using S = Smem<KP, REVERSE, KEEP>;
  constexpr int ST = S::kStages, WB = S::kW2, PANELS = KP / 64;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t base = smem_u32(smem);
  Weights* weights = reinterpret_cast<Weights*>(smem + S::kWeights);
  Bars& bar = *reinterpret_cast<Bars*>(smem + S::kBars);
  volatile int* abort = &bar.abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int vtiles = (p.V + VT - 1) / VT;
  const int vt = blockIdx.x % vtiles, piece = blockIdx.y + p.first_piece;
  const long long pair = blockIdx.x / vtiles;
  const int n = (int)(pair % p.N);
  const long long b = pair / p.N;
  const int head = (int)((long long)n * p.Nqk / p.N);
  const int chunks = ssm_chunks(p.T);
  const int first = piece * p.per, count = min(chunks, first + p.per) - first;
  const int v0 = vt * VT, vw = min(VT, p.V - v0);
  const size_t plane = (size_t)p.K * p.V;
  auto chunk_at = [&](int i) { return REVERSE ? first + count - 1 - i : first + i; };

  if (tid == 0) {
    for (int i = 0; i < 3; ++i) mbar_init(&bar.full[i], 1), mbar_init(&bar.empty[i], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&bar.gate[i], 1), mbar_init(&bar.gate_free[i], 8);
    for (int i = 0; i < 2; ++i) mbar_init(&bar.u[i], 1), mbar_init(&bar.u_free[i], 8), mbar_init(&bar.w[i], 8);
    mbar_init(&bar.put, 8), mbar_init(&bar.put_free, 1), mbar_init(&bar.hs, 1), mbar_init(&bar.hs_free, 8);
    bar.abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc(&bar.tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;
  auto stage = [&](int i) { return base + i % ST * S::kStage; };
  const int quarter = warp & 3, row = 32 * quarter + lane, half = (warp >> 2) & 1;
  const uint32_t t_lane = tmem + ((uint32_t)(32 * quarter) << 16);
  bool ok = true;
  auto wait = [&](uint64_t& b, int i) {
    if (ok) ok = warp_wait(&b, (uint32_t)i & 1u, abort);
    return ok;
  };

  if (warp < kWarpState) {  // --------------------------------------- weighted y
    for (int i = 0; i < count; ++i) {
      if (i >= WB) wait(bar.u[i % WB], i / WB - 1);  // the product that read the place's last
      wait(bar.gate[i & 3], i >> 2);
      if (!wait(bar.full[i % ST], i / ST)) break;
      const float w = weights[i & 3].w[row];
      const float2 w2 = make_float2(w, w);
      const uint32_t to = base + S::kW + i % WB * 2 * S::kY;
#pragma unroll 2
      for (int c = 0; c < 4; ++c) {
        const uint32_t at = tile_at(0, row, 4 * half + c);
        float2 f[4];
        uint32_t hi[4], lo[4];
        unpack8(ld_shared_v4(stage(i) + S::kX + at), f);
#pragma unroll
        for (int e = 0; e < 4; ++e) split_bf16x2(mul2(f[e], w2), hi[e], lo[e]);
        st_shared_v4(to + at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
        st_shared_v4(to + S::kY + at, make_uint4(lo[0], lo[1], lo[2], lo[3]));
      }
      fence_proxy_async_smem();
      warp_arrive(&bar.w[i % WB], lane);
    }
  } else if (warp < kWarpMma) {  // ---------------------------------- the state
    // This thread's row and half of the columns.  With K <= 64 the product has 64 rows, 16 in each
    // quarter's first lanes.
    constexpr int HC = VT / 2;
    const int hcol = HC * half;
    const int hrow = KP > 64 ? row : 16 * quarter + lane;
    const bool has_row = (KP > 64 || lane < 16) && hrow < p.K;
    const size_t at = (size_t)hrow * p.V + v0 + hcol;  // within [K][V]
    const float* src = p.from_state ? p.from_state + ((size_t)pair * p.pieces + piece) * plane
                       : p.from     ? p.from + pair * plane
                                    : nullptr;
    float2 H[HC / 2];
    auto given = [&](int c) { return src && has_row && hcol + c < vw ? src[at + c] : 0.f; };
#pragma unroll
    for (int c = 0; c < HC / 2; ++c) H[c] = make_float2(given(2 * c), given(2 * c + 1));
    float decay = 0.f;
    for (int i = 0; i <= count; ++i) {
      // The state before chunk i (of this order; forwards, the last state too) to its tile;
      // backwards its product with H as well.
      if (KEEP && (i < count || (!REVERSE && first + count == chunks))) {
        if (i > 0 && !wait(bar.put_free, i - 1)) break;
        if (REVERSE && !wait(bar.hs, i)) break;
        float2 d2 = make_float2(0.f, 0.f);
        if (KP > 64 || lane < 16) {
#pragma unroll
          for (int c = 0; c < HC / 8; ++c) {
            const uint32_t o = tile_at(0, hrow, hcol / 8 + c);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split_bf16x2(H[4 * c + e], hi[e], lo[e]);
            st_shared_v4(base + S::kKept + o, make_uint4(hi[0], hi[1], hi[2], hi[3]));
            st_shared_v4(base + S::kKept + KP * VT * 2 + o, make_uint4(lo[0], lo[1], lo[2], lo[3]));
            if (REVERSE) {
              float2 x[4], y[4];
              unpack8(ld_shared_v4(base + S::kHs + o), x);
              unpack8(ld_shared_v4(base + S::kHs + KP * VT * 2 + o), y);
#pragma unroll
              for (int e = 0; e < 4; ++e) d2 = fma2(H[4 * c + e], add2(x[e], y[e]), d2);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bar.put);
          if (REVERSE) mbar_arrive(&bar.hs_free);
        }
        if (REVERSE) {
          float dot = d2.x + d2.y;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(~0u, dot, o);
          if (lane == 0) p.dots[(((size_t)pair * chunks + chunk_at(i)) * vtiles + vt) * 8 + warp - kWarpState] = dot;
        }
      }
      if (i == count) break;
      wait(bar.gate[i & 3], i >> 2);
      if (!wait(bar.u[i % WB], i / WB)) break;
      tc_fence_after();
      const float total = weights[i & 3].total;
      decay += total;
      const float e = exp2_approx(total);
      const float2 e2 = make_float2(e, e);
      const uint32_t tu = t_lane + i % WB * 2 * VT + hcol;
#pragma unroll
      for (int x = 0; x < HC / 16; ++x) {
        float hi[16], lo[16];
        tmem_ld16_nowait(tu + 16 * x, hi);
        tmem_ld16_nowait(tu + VT + 16 * x, lo);
        tmem_ready(hi, lo);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          H[8 * x + c] = fma2(e2, H[8 * x + c], add2(make_float2(hi[2 * c], hi[2 * c + 1]),
                                                     make_float2(lo[2 * c], lo[2 * c + 1])));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar.u_free[i % WB]);
        mbar_arrive(&bar.gate_free[i & 3]);
      }
    }
    if (ok) {
      if (!KEEP && p.decay && vt == 0 && warp == kWarpState && lane == 0) p.decay[pair * p.pieces + piece] = decay;
      float* dst = p.to_state                         ? p.to_state + ((size_t)pair * p.pieces + piece) * plane
                   : p.to && (REVERSE ? first == 0 : first + count == chunks) ? p.to + pair * plane
                                                                              : nullptr;
      if (dst && has_row) {
#pragma unroll
        for (int c = 0; c < HC; ++c)
          if (hcol + c < vw) dst[at + c] = c & 1 ? H[c / 2].y : H[c / 2].x;
      }
    }
  } else if (warp == kWarpMma) {  // --------------------------------- products
    const uint32_t idesc = umma_idesc_bf16_ab(KP, 2 * VT, true, true);
    const bool leader = lane == 0;
    // A kept state to memory, state `chunk` of the sequence forwards, after chunk `chunk` backwards.
    auto send = [&](int i) {
      if (!wait(bar.put, i)) return false;
      const int chunk = REVERSE ? chunk_at(i) : first + i;
      if (tma) {
        for (int x = 0; x < 2; ++x)
          tma_store_4d_if(leader, &map_kept, base + S::kKept + x * KP * VT * 2, v0, 0, 2 * chunk + x, (int)pair);
        if (leader) {
          bulk_commit_group();
        }
      } else {
        uint16_t* to = p.kept + ((size_t)pair * (REVERSE ? chunks : chunks + 1) + chunk) * 2 * plane + v0;
        for (int id = lane; id < 2 * KP * VT; id += 32) {
          const int x = id / (KP * VT), r = id / VT % KP, c = id % VT;
          if (r < p.K && c < vw) {
            const uint32_t u = ld_shared_u32(tile_at(base + S::kKept + x * KP * VT * 2, r, c >> 3) + (c & 6) * 2);
            to[x * plane + (size_t)r * p.V + c] = (uint16_t)(c & 1 ? u >> 16 : u);
          }
        }
      }
      return true;
    };
    auto sent = [&]() {  // its tile may be written again
      if (leader) bulk_wait_group_read<0>();
      warp_arrive(&bar.put_free, lane);
    };
    for (int i = 0; i < count; ++i) {
      if (i >= WB) wait(bar.u_free[i % WB], i / WB - 1);
      wait(bar.full[i % ST], i / ST);
      if (!wait(bar.w[i % WB], i / WB)) break;
      tc_fence_after();
      umma_steps<L / 16, 128, 128>(leader, tmem + i % WB * 2 * VT, desc_mn(stage(i), L),
                                   desc_mn(base + S::kW + i % WB * 2 * S::kY, L), idesc, false);
      umma_commit_if(leader, &bar.u[i % WB]);
      umma_commit_if(leader, &bar.empty[i % ST]);
      if (KEEP && i > 0) sent();  // while the product runs
      if (KEEP && !send(i)) break;
    }
    if (KEEP && ok && !REVERSE && first + count == chunks) {
      if (count > 0) sent();
      send(count);
    }
    if (KEEP && leader) bulk_wait_group<0>();
  } else if (warp == kWarpLoad) {  // -------------------------------- loads
    for (int i = 0; i < count; ++i) {
      if (i >= ST && !wait(bar.empty[i % ST], i / ST - 1)) break;
      const int t0 = chunk_at(i) * L;
      if (tma) {
        if (lane == 0) {
          uint64_t* full = &bar.full[i % ST];
          unsigned char* to = smem + i % ST * S::kStage;
          mbar_arrive_expect_tx(full, S::kStage);
#pragma unroll
          for (int x = 0; x < PANELS; ++x)
            tma_load_4d(to + panel(x, L), &map_x, full, 64 * x, head, t0, (int)b);
          tma_load_4d(to + S::kX, &map_y, full, v0, n, t0, (int)b);
          if (i + 2 < count) {  // on its way to L2, before its place is free
            const int t2 = chunk_at(i + 2) * L;
#pragma unroll
            for (int x = 0; x < PANELS; ++x) tma_prefetch_4d(&map_x, 64 * x, head, t2, (int)b);
            tma_prefetch_4d(&map_y, v0, n, t2, (int)b);
            if (KEEP && REVERSE)
              for (int x = 0; x < 2; ++x) tma_prefetch_4d(&map_hs, v0, 0, 2 * chunk_at(i + 2) + x, (int)pair);
          }
        }
        __syncwarp();
      } else {
        const int rows = min(L, p.T - t0);
        const uint16_t* x0 = p.x + b * p.sx.batch + t0 * p.sx.token + (long long)head * p.K;
        for (int x = 0; x < PANELS; ++x)
          copy_tokens(stage(i) + panel(x, L), x0 + 64 * x, p.sx.token, rows, p.K - 64 * x, lane);
        copy_tokens(stage(i) + S::kX, p.y + b * p.sy.batch + t0 * p.sy.token + (long long)n * p.V + v0, p.sy.token,
                    rows, vw, lane);
        fence_proxy_async_smem();
        warp_arrive(&bar.full[i % ST], lane);
      }
      if (KEEP && REVERSE) {
        if (i > 0 && !wait(bar.hs_free, i - 1)) break;
        if (tma) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&bar.hs, 2 * KP * VT * 2);
            for (int x = 0; x < 2; ++x)
              tma_load_4d(smem + S::kHs + x * KP * VT * 2, &map_hs, &bar.hs, v0, 0, 2 * chunk_at(i) + x, (int)pair);
          }
          __syncwarp();
        } else {
          copy_state<KP>(base + S::kHs, p.Hs + ((size_t)pair * (chunks + 1) + chunk_at(i)) * 2 * plane + v0, p.K, p.V, vw,
                         lane);
          warp_arrive(&bar.hs, lane);
        }
      }
    }
    if (!ok && tma && KEEP && REVERSE)
      for (int phase = 0; phase < 2; ++phase) mbar_wait_bounded(&bar.hs, phase, kWaitLimitCycles / 64);
    if (!ok && tma)  // given up: whatever was started here arrives before the block ends
      for (int s = 0; s < ST; ++s)
        for (int phase = 0; phase < 2; ++phase) mbar_wait_bounded(&bar.full[s], phase, kWaitLimitCycles / 64);
  } else {  // ------------------------------------------------------- gates
    const uint16_t* ag = p.a + b * p.sa.batch + n;
    const float alpha = p.alpha[n], beta = p.beta[n];
    auto logit = [&](int i, int e) {
      const long long t = i < count ? (long long)chunk_at(i) * L + 32 * e + lane : p.T;
      return t < p.T ? bf16_to_f(ag[t * p.sa.token]) : -INFINITY;
    };
    int i = warp - kWarpGate;
    float4 a = make_float4(logit(i, 0), logit(i, 1), logit(i, 2), logit(i, 3));
    for (; i < count; i += 2) {
      const float4 ahead = make_float4(logit(i + 2, 0), logit(i + 2, 1), logit(i + 2, 2), logit(i + 2, 3));
      if (i >= 4 && !wait(bar.gate_free[i & 3], (i >> 2) - 1)) break;
      Weights& o = weights[i & 3];
#pragma unroll 1
      for (int e = 0; e < 4; ++e) {
        const float2 g = ssm_gate(e == 0 ? a.x : e == 1 ? a.y : e == 2 ? a.z : a.w, alpha, beta);
        o.w[32 * e + lane] = g.x;
        o.l[32 * e + lane] = g.y * kLog2e;
      }
      __syncwarp();
      const float4 d = reinterpret_cast<const float4*>(o.w)[lane], c = reinterpret_cast<const float4*>(o.l)[lane];
      // Sums of log2 f up to each token (backwards) or after it (forwards), over the four tokens of
      // the lane and the lanes before (after).
      float mine = c.x + c.y + c.z + c.w, run = mine;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const float x = REVERSE ? __shfl_up_sync(~0u, run, s) : __shfl_down_sync(~0u, run, s);
        if (REVERSE ? lane >= s : lane + s < 32) run += x;
      }
      if (lane == (REVERSE ? 31 : 0)) o.total = run;
      float rest = REVERSE ? __shfl_up_sync(~0u, run, 1) : __shfl_down_sync(~0u, run, 1);
      if (lane == (REVERSE ? 0 : 31)) rest = 0.f;
      float4 w;
      if (REVERSE) {
        const float c1 = c.x + c.y, c2 = c1 + c.z;
        w = make_float4(exp2_approx(rest + c.x), exp2_approx(rest + c1), exp2_approx(rest + c2), exp2_approx(rest + (c2 + c.w)));
      } else {
        const float r1 = c.w + c.z, r0 = r1 + c.y;
        w = make_float4(d.x * exp2_approx(rest + r0), d.y * exp2_approx(rest + r1), d.z * exp2_approx(rest + c.w),
                        d.w * exp2_approx(rest));
      }
      reinterpret_cast<float4*>(o.w)[lane] = w;
      warp_arrive(&bar.gate[i & 3], lane);
      a = ahead;
    }
  }
  if (!ok && lane == 0) {
    *abort = 1;
    atomicExch(p.status, kStatusTimeout);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) tmem_dealloc(tmem, kTmemCols);
}

// starts[segment]: the state before each segment of `sub` pieces (after it, with `reverse`), from the pieces'
// own sums and decays, chained from `from` on.
__global__ void __launch_bounds__(256)
    ssm_join_kernel(const float* __restrict__ from, const float* __restrict__ state, const float* __restrict__ decays,
                    float* __restrict__ starts, int segments, int sub, int kv, int reverse) {
  const int i = blockIdx.x * 256 + threadIdx.x, pieces = segments * sub, used = pieces - sub + 1;
  const long long pair = blockIdx.y;
  if (i >= kv) return;
  float h = from ? from[(size_t)pair * kv + i] : 0.f;
  const float* s = state + (size_t)pair * pieces * kv + i;
  const float* d = decays + pair * pieces;
  float* to = starts + (size_t)pair * segments * kv + i;
  constexpr int kAhead = 8;  // pieces loaded at once
  for (int j = 0; j < used; j += kAhead) {
    float own[kAhead], decay[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (j + u + 1 < used) {
        const int at = reverse ? pieces - 1 - j - u : j + u;
        own[u] = s[(size_t)at * kv];
        decay[u] = d[at];
      }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (j + u < used && (j + u) % sub == 0) {
        const int segment = (j + u) / sub;
        to[(size_t)(reverse ? segments - 1 - segment : segment) * kv] = h;
      }
      if (j + u + 1 < used) h = fmaf(exp2_approx(decay[u]), h, own[u]);
    }
  }
}

template <int KP, bool REVERSE, bool KEEP>
cudaError_t run(const StateProblem& p, int blocks_y, bool vec, cudaStream_t stream) {
  // At every launch: the attribute belongs to the current device.
  const cudaError_t attr =
      cudaFuncSetAttribute(ssm_state_kernel<KP, REVERSE, KEEP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Smem<KP, REVERSE, KEEP>::kBytes);
  if (attr != cudaSuccess) return attr;
  const EncodeTiledFn enc = tensor_map_encoder();
  CUtensorMap mx{}, my{}, mk{}, mh{};
  const long long pairs = (long long)p.B * p.N, chunks = ssm_chunks(p.T);
  bool tma = vec && enc && p.T > 0 && token_map(enc, &mx, p.x, p.K, p.Nqk, p.T, p.B, p.sx) &&
             token_map(enc, &my, p.y, p.V, p.N, p.T, p.B, p.sy);
  if (KEEP)
    tma = tma && state_map(enc, &mk, p.kept, p.K, p.V, 2 * (REVERSE ? chunks : chunks + 1), pairs, KP) &&
          (!REVERSE || state_map(enc, &mh, p.Hs, p.K, p.V, 2 * (chunks + 1), pairs, KP));
  const unsigned units = (unsigned)(pairs * ((p.V + VT - 1) / VT));
  ssm_state_kernel<KP, REVERSE, KEEP>
      <<<dim3(units, blocks_y), kThreads, Smem<KP, REVERSE, KEEP>::kBytes, stream>>>(mx, my, mk, mh, p, tma);
  return cudaGetLastError();
}

template <bool REVERSE, bool KEEP>
cudaError_t run_any(const StateProblem& p, int blocks_y, bool vec, cudaStream_t stream) {
  return p.K <= 64 ? run<64, REVERSE, KEEP>(p, blocks_y, vec, stream) : run<128, REVERSE, KEEP>(p, blocks_y, vec, stream);
}

}  // namespace

constexpr int kSms = 152;
static long long cut_units(int B, int N, int V) { return (long long)B * N * ((V + VT - 1) / VT); }

// Pieces of a segment for the launch that finds the segments' states: as many as make the fewest rounds
// of chunks (and three for a piece's start and end) over the SMs.  65536 tokens and 32 pairs and tiles:
// three segments' states in nine pieces, 288 blocks of 43 chunks (87 us), not 96 of 128 (112 us).
static int pieces_of(int segments, int per, long long units, bool whole) {
  long long best = 0;
  int sub = 1;
  for (int s = 1; s <= 8 && s <= per; ++s) {
    if (whole && per % s != 0) continue;
    const long long rounds = (units * (segments - 1) * s + kSms - 1) / kSms, cost = rounds * ((per + s - 1) / s + 3);
    if (best == 0 || cost < best) best = cost, sub = s;
  }
  return sub;
}

// Whole segments for every SM at most, of at least two chunks and a multiple of their pieces.
SsmCut ssm_cut(int B, int T, int N, int V) {
  const long long units = cut_units(B, N, V);
  const int chunks = ssm_chunks(T);
  SsmCut c{1, chunks > 0 ? chunks : 1};
  long long want = kSms / units;
  if (want > chunks / 2) want = chunks / 2;
  if (want < 2) return c;
  c.per = (int)((chunks + want - 1) / want);
  const int sub = pieces_of((int)want, c.per, units, false);
  c.per = (c.per + sub - 1) / sub * sub;
  c.segments = (chunks + c.per - 1) / c.per;
  return c;
}

size_t ssm_segment_floats(const SsmCut& c, int B, int N, int K, int V) {
  if (c.segments <= 1) return 0;
  const size_t state = (size_t)K * V;
  return (size_t)B * N * c.segments * (state + pieces_of(c.segments, c.per, cut_units(B, N, V), true) * (state + 1));
}

cudaError_t launch_ssm_segments(StateProblem p, const SsmCut& c, bool reverse, bool vec, float* ws,
                                cudaStream_t stream) {
  const long long pairs = (long long)p.B * p.N;
  const int kv = p.K * p.V;
  const float* from = p.from;
  p.from = nullptr;
  p.from_state = nullptr;
  p.kept = nullptr;
  const int sub = pieces_of(c.segments, c.per, cut_units(p.B, p.N, p.V), true);
  p.pieces = c.segments * sub;
  p.per = c.per / sub;
  p.first_piece = reverse ? sub : 0;  // the last segment of the order ends the sequence: not needed
  p.to_state = ws + (size_t)pairs * c.segments * kv;
  p.decay = p.to_state + (size_t)pairs * p.pieces * kv;
  const cudaError_t err = reverse ? run_any<true, false>(p, (c.segments - 1) * sub, vec, stream)
                                  : run_any<false, false>(p, (c.segments - 1) * sub, vec, stream);
  if (err != cudaSuccess) return err;
  ssm_join_kernel<<<dim3((kv + 255) / 256, (unsigned)pairs), 256, 0, stream>>>(from, p.to_state, p.decay, ws,
                                                                               c.segments, sub, kv, reverse);
  return cudaGetLastError();
}

cudaError_t launch_ssm_kept_states(StateProblem p, const SsmCut& c, bool reverse, bool vec, cudaStream_t stream) {
  p.pieces = c.segments;
  p.per = c.per;
  p.first_piece = 0;
  p.to_state = nullptr;
  p.decay = nullptr;
  return reverse ? run_any<true, true>(p, c.segments, vec, stream) : run_any<false, true>(p, c.segments, vec, stream);
}

}  // namespace m2rnn
