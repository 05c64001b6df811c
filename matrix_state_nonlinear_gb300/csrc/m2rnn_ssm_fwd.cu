// m2rnn_ssm_fwd.cu — the selective scan of a prompt in chunks of 128 tokens (see include/m2rnn.h).
//
// With c_t the sum of log f over a chunk up to token t, and H the state before the chunk,
//   y_t = exp(c_t) H^T q_t + sum_{s <= t} exp(c_t - c_s) d_s (q_t . k_s) v_s + w_r v_t
//   H  <- exp(c_127) H + sum_s k_s (exp(c_127 - c_s) d_s v_s)^T
// so that a chunk is four products on the 5th-generation tensor cores, a token per tensor-memory
// lane: S = q k^T, Y1 = q H, Y2 = P v (P = S decayed and masked), U = k^T (weighted v).
// One block walks the chunks of one (batch, head) pair and one tile of 64 value columns.  Its warps
// hand each other work through mbarriers, so that several chunks are in flight at once:
//   8 warps   P from S and the weighted v (a quarter of the tokens and half the columns each);
//   8 warps   y from Y1, Y2 and v (half the columns each);
//   8 warps   the state, float32 in registers (half the columns each);
//   2 warps   issue the products: S and P v; q H and U;
//   2 warps   load the tiles (TMA) and compute the gates of every other chunk.
//  * S is decayed in float32 and rounded to bf16 in tensor memory, the first operand of P v; H is
//    rounded to bf16 as an operand; y is bf16.  The state itself is float32 and takes U with float32
//    weights: the weighted v enters as two bf16 values (17 bits), two products.
//  * exp(c_t - c_s) is split at the end of s's block of 32, exp(c_t - c_end) exp(c_end - c_s), two
//    factors of at most one: one exponential per row and block instead of one per score.  No sum in an
//    exponent runs over more than a block, and where one is large it is kept in two parts (ChunkGates).
//  * Only H -> q H and U -> H follow the sequence; S and U of the next chunk are issued before this
//    chunk's P v, so that P never waits for the tensor cores' latency.
//  * q and k have their own stages, free as soon as the products have read them: with K = 128 only two
//    fit, and held until y was out they left the loads in the open (222 -> 165 us for 4 sequences of
//    8192 tokens and 32 heads).  y leaves through v's place.
//  * The warps run five different programs, together near the instruction cache's size, so each is
//    kept short: waits that do not succeed at once share one function, loads have one site each, and
//    P's loop of four is unrolled by two (246 us for 8 x 16384; by one 256, by four, before the weights were taken
//    by block, 287 instead of 240).
// Where the pairs are fewer than the SMs, segments of a sequence run side by side
// (m2rnn_ssm_state.cu).
// Measured: 246 us for 8 x 16384 tokens of 16 heads, K = V = 64 (4.4 TB/s, 65 % of a copy), 244 us for
// 65536 tokens of 16 heads, V = 128, after their segments' states, 152 us for 4 x 8192 tokens of 32
// heads, K = 128.  A chunk is 8700 warp instructions and about 3800 cycles with K = 64; they issue in 58 %
// of the slots.  The warps of P bound it, which decay S and weigh v element by element, and the waits
// between roles.  Weighing v in the state's warps took 287 us or more instead of 264, in four of the eight
// warps 290 instead of 282 (8 x 16384, before the loops were unrolled).
#include "m2rnn_ssm_tc.cuh"

namespace m2rnn {
namespace {

constexpr int L = kTokens;
constexpr int VT = kSsmColumns;
// First warp of each kind.
constexpr int kWarpY = 8, kWarpState = 16, kWarpMma = 24, kWarpLoad = 26, kWarps = 28;
constexpr int kThreads = 32 * kWarps;

// Tensor memory columns.  S has two buffers, and P takes the place of its S: the 64 columns of
// scores that a warp reads become 32 columns of bf16 pairs at their start.  U is in two halves, of
// the high and the low parts of the weighted v.
constexpr int kColS = 0, kColY1 = 256, kColY2 = 320, kColU = 384, kTmemCols = 512;

template <int KP>
struct Smem {
  static constexpr int kStages = KP <= 64 ? 3 : 2, kStagesV = KP <= 64 ? 4 : 2;
  static constexpr int kQ = L * KP * 2, kV = L * VT * 2;
  static constexpr int kStage = 2 * kQ;  // q and k
  static constexpr int kVs = kStages * kStage;
  static constexpr int kW = kVs + kStagesV * kV;  // weighted v, high and low
  static constexpr int kH = kW + 2 * kV;
  static constexpr int kGates = kH + KP * VT * 2;
  static constexpr int kWr = kGates + 4 * (int)sizeof(ChunkGates);
  static constexpr int kBars = kWr + VT * 4;
  static constexpr int kBytes = kBars + 320 + 1024;  // and slack to align the tiles
  static_assert(kBytes <= 227 * 1024 && sizeof(ChunkGates) % 16 == 0, "");
};

// A barrier's next phase completes only after every waiter has passed the phase before (a waiter
// two phases behind would mistake one for the other).  Where a chunk's work may run that far
// ahead there is a barrier for every buffer, stage or slot.
struct Bars {
  uint64_t full[3], empty[3];      // q and k of a stage: loaded; done with (S, q H and U are)
  uint64_t vfull[4], vempty[4];    // v of a stage: loaded; done with (by the warps of y)
  uint64_t gate[4], gate_free[4];  // gates of a chunk: written; done with (by y and the state)
  uint64_t s[2], p[2];             // S, P, by buffer
  uint64_t y, y_free;              // q H and P v done; Y read
  uint64_t u, u_free, w, h;        // U done, read; weighted v, H done
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Bars) <= 320, "");

// P from S for the half of the columns with the rows' own block, where that block's tokens differ in hi: as
// below, but its weights are taken part by part.  Few blocks decay so far; inside the usual loop, which is
// at the edge of the instruction cache, the same cost every block 255 to 290 us instead of 246 (8 x 16384).
static __device__ __noinline__ void put_wide_scores(uint32_t ts, const ChunkGates& G, int row, int half) {
  const int quarter = row >> 5;
  const float hi = G.hi[row], lo = G.lo[row];
#pragma unroll 1
  for (int x = 0; x < 4; ++x) {
    const int cb = 2 * half + (x >> 1), col = 32 * cb + 16 * (x & 1);
    float s[16];
    uint32_t out[8];
    tmem_ld16_nowait(ts + col, s);
    tmem_ready(s);
    const float u = cb < quarter ? exp2_approx((hi + lo) + G.span[quarter][cb + 1]) : 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float q[2];
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int k = 2 * e + z;
        const float m = cb < quarter ? u * G.wd[col + k] : exp2_approx((hi - G.hi[col + k]) + (lo - G.diag[col + k]));
        q[z] = col + k <= row ? s[k] * m : 0.f;
      }
      out[e] = pack_bf16x2(q[0], q[1]);
    }
    tmem_st8(ts + 64 * half + 8 * x, out);
  }
}

template <int KP>
__global__ void __launch_bounds__(kThreads, 1)
    ssm_forward_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, SsmProblem p, SsmCut cut, bool tma, bool vec) {
  using S = Smem<KP>;
  constexpr int ST = S::kStages, SV = S::kStagesV, PANELS = KP / 64;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t base = smem_u32(smem);
  ChunkGates* gates = reinterpret_cast<ChunkGates*>(smem + S::kGates);
  float* wr = reinterpret_cast<float*>(smem + S::kWr);
  Bars& bar = *reinterpret_cast<Bars*>(smem + S::kBars);
  volatile int* abort = &bar.abort;
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
    for (int i = 0; i < 3; ++i) mbar_init(&bar.full[i], 1), mbar_init(&bar.empty[i], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&bar.vfull[i], 1), mbar_init(&bar.vempty[i], 8);
    for (int i = 0; i < 4; ++i) mbar_init(&bar.gate[i], 1), mbar_init(&bar.gate_free[i], 16);
    for (int i = 0; i < 2; ++i) mbar_init(&bar.s[i], 1), mbar_init(&bar.p[i], 8);
    mbar_init(&bar.y, 2);
    mbar_init(&bar.y_free, 8), mbar_init(&bar.u, 1), mbar_init(&bar.u_free, 8);
    mbar_init(&bar.w, 8), mbar_init(&bar.h, 8);
    bar.abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc(&bar.tmem, kTmemCols);
  if (tid < VT) wr[tid] = tid < vw ? p.w_r[(size_t)n * p.V + v0 + tid] : 0.f;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;
  auto stage = [&](int i) { return base + i % ST * S::kStage; };
  auto vstage = [&](int i) { return base + S::kVs + i % SV * S::kV; };
  const int quarter = warp & 3, row = 32 * quarter + lane;  // token of the chunk, tensor-memory lane
  const uint32_t t_lane = tmem + ((uint32_t)(32 * quarter) << 16);
  bool ok = true;  // uniform in the warp
  auto wait = [&](uint64_t& b, int i) {
    if (ok) ok = warp_wait(&b, (uint32_t)i & 1u, abort);
    return ok;
  };

  if (warp < kWarpY) {  // ------------------------------------------- P from S
    const int half = warp >> 2;
    // Half a token's v of chunk i, weighted, as two bf16 values.
    auto put_weighted = [&](int i) {
      if (i > 0) wait(bar.u, i - 1);  // the product that read it
      wait(bar.gate[i & 3], i >> 2);
      if (!wait(bar.vfull[i % SV], i / SV)) return;
      const float w = gates[i & 3].wk[row];
      const float2 w2 = make_float2(w, w);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t at = tile_at(0, row, 4 * half + c);
        float2 f[4];
        uint32_t hi[4], lo[4];
        unpack8(ld_shared_v4(vstage(i) + at), f);
#pragma unroll
        for (int e = 0; e < 4; ++e) split_bf16x2(mul2(f[e], w2), hi[e], lo[e]);
        st_shared_v4(base + S::kW + at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
        st_shared_v4(base + S::kW + S::kV + at, make_uint4(lo[0], lo[1], lo[2], lo[3]));
      }
      fence_proxy_async_smem();
      warp_arrive(&bar.w, lane);
    };
    if (count > 0) put_weighted(0);
    for (int i = 0; i < count && ok; ++i) {
      const ChunkGates& G = gates[i & 3];  // (waited for with v)
      const float own = G.hi[row] + G.lo[row];
      const bool wide = half == quarter >> 1 && G.wide(quarter);
      if (!wait(bar.s[i & 1], i >> 1)) break;
      tc_fence_after();
      const uint32_t ts = t_lane + kColS + (i & 1) * 128;
      // Block cb of 32 columns against the quarter's own block of 32 rows, 16 columns at a time.
      if (wide) {
        put_wide_scores(ts, G, row, half);
      } else {
#pragma unroll 2
        for (int x = 0; x < 4; ++x) {
          const int cb = 2 * half + (x >> 1), col = 32 * cb + 16 * (x & 1);
          uint32_t out[8];
          if (cb > quarter) {
#pragma unroll
            for (int e = 0; e < 8; ++e) out[e] = 0u;
          } else {
            float s[16];
            tmem_ld16_nowait(ts + col, s);
            if (cb < quarter) {
              const float u = exp2_approx(own + G.span[quarter][cb + 1]);
              const float2 u2 = make_float2(u, u);
              const float4* w = reinterpret_cast<const float4*>(G.wd + col);
              tmem_ready(s);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float4 wv = w[e];
                const float2 a = mul2(make_float2(s[4 * e], s[4 * e + 1]), mul2(u2, make_float2(wv.x, wv.y)));
                const float2 c = mul2(make_float2(s[4 * e + 2], s[4 * e + 3]), mul2(u2, make_float2(wv.z, wv.w)));
                out[2 * e] = pack_bf16x2(a.x, a.y);
                out[2 * e + 1] = pack_bf16x2(c.x, c.y);
              }
            } else {
              const float4* w = reinterpret_cast<const float4*>(G.diag + col);
              tmem_ready(s);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float4 wv = w[e];
                const float m[4] = {exp2_approx(own - wv.x), exp2_approx(own - wv.y), exp2_approx(own - wv.z),
                                    exp2_approx(own - wv.w)};
                float q[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) q[z] = 16 * (x & 1) + 4 * e + z <= lane ? s[4 * e + z] * m[z] : 0.f;
                out[2 * e] = pack_bf16x2(q[0], q[1]);
                out[2 * e + 1] = pack_bf16x2(q[2], q[3]);
              }
            }
          }
          tmem_st8(ts + 64 * half + 8 * x, out);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(&bar.p[i & 1], lane);
      if (i + 1 < count) put_weighted(i + 1);
    }
  } else if (warp < kWarpState) {  // ----------------------------------- y
    const int half = (warp - kWarpY) >> 2;
    const long long ystride = (long long)p.N * p.V;
    for (int i = 0; i < count; ++i) {
      if (!wait(bar.y, i)) break;  // (P's warps had the gates)
      tc_fence_after();
      const float e = exp2_approx(gates[i & 3].from_start(row));
      const float2 e2 = make_float2(e, e);
      const uint32_t tv = vstage(i);
#pragma unroll 1
      for (int x = 2 * half; x < 2 * half + 2; ++x) {  // 16 columns at a time, in place of this token's v
        float y1[16], y2[16];
        tmem_ld16_nowait(t_lane + kColY1 + 16 * x, y1);
        tmem_ld16_nowait(t_lane + kColY2 + 16 * x, y2);
        const uint4 va = ld_shared_v4(tile_at(tv, row, 2 * x)), vb = ld_shared_v4(tile_at(tv, row, 2 * x + 1));
        const float4* w4 = reinterpret_cast<const float4*>(wr + 16 * x);
        tmem_ready(y1, y2);
        if (x & 1) {
          tc_fence_before();
          warp_arrive(&bar.y_free, lane);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float2 v[4];
          uint32_t o[4];
          unpack8(c ? vb : va, v);
          const float4 w0 = w4[2 * c], w1 = w4[2 * c + 1];
          const float2 w[4] = {make_float2(w0.x, w0.y), make_float2(w0.z, w0.w), make_float2(w1.x, w1.y),
                               make_float2(w1.z, w1.w)};
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const int k = 8 * c + 2 * z;
            const float2 r = fma2(w[z], v[z], fma2(e2, make_float2(y1[k], y1[k + 1]), make_float2(y2[k], y2[k + 1])));
            o[z] = pack_bf16x2(r.x, r.y);
          }
          st_shared_v4(tile_at(tv, row, 2 * x + c), make_uint4(o[0], o[1], o[2], o[3]));
        }
      }
      __syncwarp();
      const int t0 = (first + i) * L + 32 * quarter, left = min(32, p.T - t0), col0 = 32 * half;
      uint16_t* yg = p.y + ((b * p.T + t0) * p.N + n) * p.V + v0 + col0;
      if (vec) {  // 64 contiguous bytes of eight tokens at a time
        const int ch = lane & 3, most = col0 + ch * 8 < vw ? left : 0;
        uint16_t* to = yg + (lane >> 2) * ystride + ch * 8;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = (lane >> 2) + 8 * x;
          if (r < most) *reinterpret_cast<uint4*>(to) = ld_shared_v4(tile_at(tv, 32 * quarter + r, 4 * half + ch));
          to += 8 * ystride;
        }
      } else {
        for (int x = lane; x < 32 * 32; x += 32) {
          const int r = x >> 5, col = x & 31;
          if (r < left && col0 + col < vw) {
            const uint32_t u = ld_shared_u32(tile_at(tv, 32 * quarter + r, 4 * half + (col >> 3)) + (col & 6) * 2);
            yg[r * ystride + col] = (uint16_t)(col & 1 ? u >> 16 : u);
          }
        }
      }
      fence_proxy_async_smem();  // the rows are the next load's
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar.vempty[i % SV]);
        mbar_arrive(&bar.gate_free[i & 3]);
      }
    }
  } else if (warp < kWarpMma) {  // ------------------------------------- the state
    // This thread's row of the state.  With K <= 64 the product has 64 rows, 16 in each quarter's
    // first lanes.
    const int hrow = KP > 64 ? row : 16 * quarter + lane;
    const bool has_row = (KP > 64 || lane < 16) && hrow < p.K;
    constexpr int HC = VT / 2;  // this thread's columns, from hcol
    const int hcol = HC * ((warp - kWarpState) >> 2);
    float2 H[HC / 2];
    const float* src = cut.segments > 1 ? p.ws + ((size_t)pair * cut.segments + seg) * plane
                       : p.H0           ? p.H0 + pair * plane
                                        : nullptr;
    auto first_state = [&](int c) {
      return src && has_row && hcol + c < vw ? src[(size_t)hrow * p.V + v0 + hcol + c] : 0.f;
    };
#pragma unroll
    for (int c = 0; c < HC / 2; ++c) H[c] = make_float2(first_state(2 * c), first_state(2 * c + 1));
    // The state as the next product's bf16 operand.
    auto put_state = [&]() {
      if (KP <= 64 && lane >= 16) return;
#pragma unroll
      for (int c = 0; c < HC / 8; ++c) {
        uint32_t hi[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) hi[e] = pack_bf16x2(H[4 * c + e].x, H[4 * c + e].y);
        st_shared_v4(tile_at(base + S::kH, hrow, hcol / 8 + c), make_uint4(hi[0], hi[1], hi[2], hi[3]));
      }
    };
    put_state();
    fence_proxy_async_smem();
    warp_arrive(&bar.h, lane);
    for (int i = 0; i < count; ++i) {
      if (!wait(bar.u, i)) break;  // (weighing v took the gates)
      tc_fence_after();
      const float e = exp2_approx(gates[i & 3].total());
      const float2 e2 = make_float2(e, e);
#pragma unroll
      for (int x = 0; x < HC / 16; ++x) {
        float hi[16], lo[16];
        tmem_ld16_nowait(t_lane + kColU + hcol + 16 * x, hi);
        tmem_ld16_nowait(t_lane + kColU + VT + hcol + 16 * x, lo);
        tmem_ready(hi, lo);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          H[8 * x + c] = fma2(e2, H[8 * x + c], add2(make_float2(hi[2 * c], hi[2 * c + 1]),
                                                     make_float2(lo[2 * c], lo[2 * c + 1])));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar.u_free);
        mbar_arrive(&bar.gate_free[i & 3]);
      }
      if (!wait(bar.empty[i % ST], i / ST)) break;  // q H of this chunk still reads the state's tile
      put_state();
      fence_proxy_async_smem();
      warp_arrive(&bar.h, lane);
    }
    if (ok && p.H_T && first + count == chunks && has_row) {
      float* dst = p.H_T + pair * plane + (size_t)hrow * p.V + v0 + hcol;
#pragma unroll
      for (int c = 0; c < HC; ++c)
        if (hcol + c < vw) dst[c] = c & 1 ? H[c / 2].y : H[c / 2].x;
    }
  } else if (warp < kWarpLoad) {  // ------------------------------------ products
    const uint32_t idesc_y = umma_idesc_bf16_ab(128, VT, false, true);
    const bool leader = lane == 0;
    if (warp == kWarpMma) {
      // S of chunk i + 1 into the buffer of P of chunk i - 1, then P v of chunk i.
      const uint32_t idesc_s = umma_idesc_bf16(128, 128, false);
      for (int i = -1; i < count; ++i) {
        const uint32_t next = stage(i + 1);
        if (i > 0) wait(bar.y, i - 1);
        if (i + 1 < count) {
          if (!wait(bar.full[(i + 1) % ST], (i + 1) / ST)) break;
          umma_steps<KP / 16, 2, 2, L * 8 - 8, L * 8 - 8>(leader, tmem + kColS + ((i + 1) & 1) * 128, desc_k(next),
                                                          desc_k(next + S::kQ), idesc_s, false);
          umma_commit_if(leader, &bar.s[(i + 1) & 1]);
        }
        if (i < 0) continue;
        if (i > 0) wait(bar.y_free, i - 1);
        wait(bar.vfull[i % SV], i / SV);
        if (!wait(bar.p[i & 1], i >> 1)) break;
        tc_fence_after();
        const uint64_t dv = desc_mn(vstage(i), L);
        const uint32_t tp = tmem + kColS + (i & 1) * 128;
        umma4_ta_if<128>(leader, tmem + kColY2, tp, dv, idesc_y, 0u);
        umma4_ta_if<128>(leader, tmem + kColY2, tp + 64, dv + 512, idesc_y, 1u);
        umma_commit_if(leader, &bar.y);
      }
    } else {
      // U of chunk i (k^T times the weighted v, high and low side by side), then q H.
      const uint32_t idesc_u = umma_idesc_bf16_ab(KP, 2 * VT, true, true);
      const uint64_t dh = desc_mn(base + S::kH, KP), dw = desc_mn(base + S::kW, L);
      for (int i = 0; i < count; ++i) {
        wait(bar.full[i % ST], i / ST);
        if (i > 0) wait(bar.u_free, i - 1);
        if (!wait(bar.w, i)) break;
        tc_fence_after();
        umma_steps<L / 16, 128, 128>(leader, tmem + kColU, desc_mn(stage(i) + S::kQ, L), dw, idesc_u, false);
        umma_commit_if(leader, &bar.u);
        if (i > 0) wait(bar.y_free, i - 1);
        wait(bar.s[i & 1], i >> 1);  // so that the stage is done with when q H is
        if (!wait(bar.h, i)) break;
        tc_fence_after();
        umma_steps<KP / 16, 2, 128, L * 8 - 8>(leader, tmem + kColY1, desc_k(stage(i)), dh, idesc_y, false);
        umma_commit_if(leader, &bar.empty[i % ST]);
        umma_commit_if(leader, &bar.y);
      }
    }
  } else {  // ---------------------------------------------------------- gates and loads
    const uint16_t* ag = p.a + b * p.sa.batch + n;
    const float alpha = p.alpha[n], beta = p.beta[n];
    // Token 32 e + lane of a chunk, loaded two chunks ahead.
    auto logit = [&](int i, int e) {
      const long long t = (long long)(first + i) * L + 32 * e + lane;
      return i < count && t < p.T ? bf16_to_f(ag[t * p.sa.token]) : -INFINITY;
    };
    int i = warp - kWarpLoad;
    float4 a = make_float4(logit(i, 0), logit(i, 1), logit(i, 2), logit(i, 3));
    for (; i < count; i += 2) {
      const float4 ahead = make_float4(logit(i + 2, 0), logit(i + 2, 1), logit(i + 2, 2), logit(i + 2, 3));
      const int t0 = (first + i) * L, s = i % ST, sv = i % SV, rows = min(L, p.T - t0);
      // q and k of a stage are free once the products have read them, v when y has left its place.
      if (i >= ST && !wait(bar.empty[s], i / ST - 1)) break;
      if (tma) {
        if (lane == 0) {
          unsigned char* to = smem + s * S::kStage;
          mbar_arrive_expect_tx(&bar.full[s], 2 * S::kQ);
#pragma unroll 1
          for (int x = 0; x < PANELS; ++x) {
            tma_load_4d(to + panel(x, L), &map_q, &bar.full[s], 64 * x, head, t0, (int)b);
            tma_load_4d(to + S::kQ + panel(x, L), &map_k, &bar.full[s], 64 * x, head, t0, (int)b);
          }
        }
        __syncwarp();
      } else {
        const uint16_t* q = p.q + b * p.sq.batch + t0 * p.sq.token + (long long)head * p.K;
        const uint16_t* k = p.k + b * p.sk.batch + t0 * p.sk.token + (long long)head * p.K;
#pragma unroll 1
        for (int x = 0; x < 2 * PANELS; ++x) {
          const int half = x / PANELS, c = x % PANELS;
          copy_tokens(stage(i) + half * S::kQ + panel(c, L), (half ? k : q) + 64 * c,
                      half ? p.sk.token : p.sq.token, rows, p.K - 64 * c, lane);
        }
        fence_proxy_async_smem();
        warp_arrive(&bar.full[s], lane);
      }
      if (i >= 4 && !wait(bar.gate_free[i & 3], (i >> 2) - 1)) break;
      put_chunk_gates(
          gates[i & 3], [&](int e) { return e == 0 ? a.x : e == 1 ? a.y : e == 2 ? a.z : a.w; }, alpha, beta, lane);
      warp_arrive(&bar.gate[i & 3], lane);
      a = ahead;
      if (i >= SV && !wait(bar.vempty[sv], i / SV - 1)) break;
      if (tma) {
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar.vfull[sv], S::kV);
          tma_load_4d(smem + S::kVs + sv * S::kV, &map_v, &bar.vfull[sv], v0, n, t0, (int)b);
          if (i + 2 < count) {  // on its way to L2, before its place is free
            const int t2 = t0 + 2 * L;
#pragma unroll 1
            for (int x = 0; x < PANELS; ++x) {
              tma_prefetch_4d(&map_q, 64 * x, head, t2, (int)b);
              tma_prefetch_4d(&map_k, 64 * x, head, t2, (int)b);
            }
            tma_prefetch_4d(&map_v, v0, n, t2, (int)b);
          }
        }
        __syncwarp();
      } else {
        copy_tokens(vstage(i), p.v + b * p.sv.batch + t0 * p.sv.token + (long long)n * p.V + v0, p.sv.token, rows, vw,
                    lane);
        fence_proxy_async_smem();
        warp_arrive(&bar.vfull[sv], lane);
      }
    }
    // Given up: whatever was started here arrives before the block ends (a stage's load that was
    // not started times out, one of an earlier chunk has long arrived).
    if (!ok && tma)
#pragma unroll 1
      for (int phase = 0; phase < 2; ++phase) {
#pragma unroll 1
        for (int s = 0; s < ST; ++s) mbar_wait_bounded(&bar.full[s], phase, kWaitLimitCycles / 64);
#pragma unroll 1
        for (int s = 0; s < SV; ++s) mbar_wait_bounded(&bar.vfull[s], phase, kWaitLimitCycles / 64);
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

template <int KP>
cudaError_t run(const SsmProblem& p, const SsmCut& cut, bool vec, cudaStream_t stream) {
  // At every launch: the attribute belongs to the current device.
  const cudaError_t attr =
      cudaFuncSetAttribute(ssm_forward_kernel<KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<KP>::kBytes);
  if (attr != cudaSuccess) return attr;
  const EncodeTiledFn enc = tensor_map_encoder();
  CUtensorMap mq{}, mk{}, mv{};
  const bool tma = vec && enc && p.T > 0 && token_map(enc, &mq, p.q, p.K, p.Nqk, p.T, p.B, p.sq) &&
                   token_map(enc, &mk, p.k, p.K, p.Nqk, p.T, p.B, p.sk) &&
                   token_map(enc, &mv, p.v, p.V, p.N, p.T, p.B, p.sv);
  const unsigned units = (unsigned)((long long)p.B * p.N * ((p.V + VT - 1) / VT));
  ssm_forward_kernel<KP><<<dim3(units, cut.segments), kThreads, Smem<KP>::kBytes, stream>>>(
      mq, mk, mv, p, cut, tma, vec);
  return cudaGetLastError();
}

}  // namespace

size_t ssm_forward_workspace_bytes(int B, int T, int N, int, int K, int V) {
  return sizeof(float) * ssm_segment_floats(ssm_cut(B, T, N, V), B, N, K, V);
}

cudaError_t launch_ssm_forward(const SsmProblem& p, cudaStream_t stream) {
  const bool vec = rows_of_16(p.q, p.sq, p.K) && rows_of_16(p.k, p.sk, p.K) && rows_of_16(p.v, p.sv, p.V) &&
                   aligned_to(p.y, 16);
  const SsmCut cut = ssm_cut(p.B, p.T, p.N, p.V);
  if (cut.segments > 1 || p.Hs) {
    StateProblem s{p.k, p.v, p.a, p.alpha, p.beta, p.sk, p.sv, p.sa, p.B, p.T, p.N, p.Nqk, p.K, p.V, p.H0};
    s.status = p.status;
    cudaError_t err = cudaSuccess;
    if (cut.segments > 1) {
      err = launch_ssm_segments(s, cut, false, vec, p.ws, stream);
      s.from_state = p.ws;
    }
    if (err == cudaSuccess && p.Hs) {
      s.kept = p.Hs;
      err = launch_ssm_kept_states(s, cut, false, vec && aligned_to(p.Hs, 16), stream);
    }
    if (err != cudaSuccess) return err;
  }
  return p.K <= 64 ? run<64>(p, cut, vec, stream) : run<128>(p, cut, vec, stream);
}

}  // namespace m2rnn
