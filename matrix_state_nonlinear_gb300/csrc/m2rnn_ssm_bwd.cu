// m2rnn_ssm_bwd.cu — gradients of the selective scan (see include/m2rnn.h).
//
// Two passes over chunks of 128 tokens.  The first (m2rnn_ssm_state.cu) runs the state's gradient
// backwards, G <- exp(c_127) G + sum_t exp(c_t) q_t dy_t^T, and keeps it after every chunk.  With G
// there and the state H before the chunk (kept by the forward), chunks are independent; the second
// pass, here, takes them in any order.  With P_ts = exp(c_t - c_s) d_s (q_t . k_s) and dS_ts the
// same of (dy_t . v_s), s <= t:
//   dq = dS k + (exp(c) dy) H^T              dk = dS^T q + (w v) G^T,   w_s = exp(c_127 - c_s) d_s
//   dv = P^T dy + w (k G) + w_r dy
// and for the gate, with E_ts = P_ts (dy_t . v_s) over s < t,
//   r_u = exp(c_u) (q_u H) . dy_u,   l_s = w_s (k_s G) . v_s,
//   g_t = dL/dlog f_t = exp(c_127) <G, H> + sum_{u >= t} r_u + sum_{s < t} l_s + sum_{u >= t > s} E_us
//   da = sigmoid (l + sum_u E_us + E_ss) / d - alpha sigmoid g,   dalpha = -sum d g,   dbeta = sum da
// g sums what passes token t, from the states and tokens before it to those after, and nothing else: every
// term has f_t in it.  (The last sum is also that of column s less row s over s < t, 31 us cheaper for the
// step below.  But what cancels there leaves 2^-24 of the chunk's larger E at the tokens that forget
// everything, where d is large: dalpha, which weighs g by d, was up to 2^-12 of its terms off.)
//
// Precision: dq, dk, dv are bf16, and one operand of each of their products is rounded to bf16 (P,
// dS, exp(c) dy, w v); H and G enter as two bf16 values each.  The gate's gradient ends in float32
// sums over all tokens: E is float32 from float32 scores, and q H, k G are float32 but for the 17
// bits of H and G.
//
// One block is resident per SM (shared memory) and walks steps: one (head, value tile) of one
// chunk.  Heads that share q and k are consecutive steps of one item, whose dq and dk add up in
// tensor memory; items of many heads may be split (float32 parts, added in a fixed order).  Splits of
// one item run side by side and read the same tokens' rows; equal stretches of all the steps per block
// would leave fewer parts (28 -> 19 us to add) but took 405 us instead of 378.
// Sixteen warps do each phase together (a row, i.e. token, per lane; 16 or 32 columns per warp),
// four others issue products, load, store, and finish the gate's gradient.  K = 128 fills tensor memory
// (S, dP, dq, dk) and shared memory, so a step's phases follow one another and that chain is what
// bounds it: 423 us for 4 x 8192 tokens of 32 heads on one q and k, K = 128, V = 64 (15100 cycles a step,
// the tensor cores busy 27 %), 37 us for 4 x 2048 of 8 heads, K = V = 64.  A small launch before
// computes every chunk's gates, and outputs leave through shared memory, whole rows at a time.
#include "m2rnn_ssm_tc.cuh"

namespace m2rnn {
namespace {

constexpr int L = kTokens;
constexpr int VT = kSsmColumns;
constexpr int kWarpMma = 16, kWarpLoad = 17, kWarpStore = 18, kWarps = 20;  // 0..15: element-wise; 19: the gate's gradient
constexpr int kThreads = 32 * kWarps;

// Tensor memory columns: q H and then P^T dy in the place of S, k G in the place of dP.
constexpr int kColDq = 0, kColDk = 128, kColS = 256, kColDp = 384, kTmemCols = 512;

// A chunk's gates in memory: what the products need, and per token sigmoid / d, alpha sigmoid, d.
struct alignas(16) BackwardGates {
  ChunkGates g;
  float rho[L], asig[L], d[L];
};
static_assert(sizeof(BackwardGates) % 16 == 0, "");

// Sums over a head's chunk, per token; parts by column group or quarter.
struct alignas(16) Sums {
  float row[4][L];   // E of a row over the blocks before its own
  float first[L];    // and over the first 16 columns of its own
  float col[4][L];   // E of a column over the rows of a later block; [its own block]: E over the pairs of the
                     // column's piece of 16 and block that its token separates
  float own[L];      // E of a column over the rows of its own block, its own included
  float row_state[4][L], col_state[4][L];
};

template <int KP>
struct Smem {
  static constexpr int kTile = L * 128;            // 128 rows of 64 values
  static constexpr int kQ = 0, kK = kQ + L * KP * 2;
  static constexpr int kV = kK + L * KP * 2, kDy = kV + kTile;
  static constexpr int kState = kDy + kTile;       // H, later G: high, low
  static constexpr int kScaled = kState + 2 * KP * VT * 2;  // exp(c) dy, later w v
  static constexpr int kP = kScaled + kTile, kDs = kP + 2 * kTile;
  static constexpr int kGates = kDs + 2 * kTile;
  static constexpr int kSums = kGates + 2 * (int)sizeof(BackwardGates);
  static constexpr int kWr = kSums + (int)sizeof(Sums);
  static constexpr int kBars = kWr + 4 * 16 * 4;
  static constexpr int kBytes = kBars + 256 + 1024;  // and slack to align the tiles
  static_assert(kBytes <= 227 * 1024 && kWr % 16 == 0, "");
};

// One phase per step (per item: qk, acc_free; per head: sums, sums_free); every barrier's next
// phase needs its waiters to have passed the one before.
struct Bars {
  uint64_t qk, vd, h, g;            // tiles loaded
  uint64_t step_free, vd_read;      // the step's accumulators, v and dy read
  uint64_t scaled1, scaled2;        // exp(c) dy, w v written
  uint64_t s, pds, hd, q_read, gd, done;  // S, dP done; P, dS written; q H done, read; k G, P^T dy done; all done
  uint64_t acc_free;                // dq, dk read
  uint64_t gate[2], gate_free[2];
  uint64_t sums, sums_free;
  uint64_t out, out_free;           // outputs in shared memory, on their way
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Bars) <= 256, "");

// The work of one block: items blockIdx.x, + gridDim.x, ...; an item is a chunk of a batch row and
// q/k head, for `heads` of its heads, each for every value tile.
struct Plan {
  int chunks, vtiles, rep, splits, per_split;
  long long items;
};
struct Workspace {
  float *segments, *dots, *par, *dqp, *dkp;
  BackwardGates* gates;
  uint16_t* G;
  size_t floats;
};

// Position in a block's list of steps.
struct Cursor {
  long long item;
  int b, group, chunk, split, head, last_head, vt;
  int item_no, head_no;
  __device__ bool start(const Plan& plan, int nqk) {
    item = blockIdx.x, item_no = 0, head_no = 0;
    return open(plan, nqk);
  }
  __device__ bool open(const Plan& plan, int nqk) {
    if (item >= plan.items) return false;
    uint32_t x = (uint32_t)item;
    split = (int)(x % plan.splits), x /= plan.splits;
    chunk = (int)(x % plan.chunks), x /= plan.chunks;
    group = (int)(x % nqk);
    b = (int)(x / nqk);
    head = group * plan.rep + split * plan.per_split;
    last_head = min(head + plan.per_split, (group + 1) * plan.rep) - 1;
    vt = 0;
    return true;
  }
  __device__ bool first(const Plan& plan) const { return vt == 0 && head == group * plan.rep + split * plan.per_split; }
  __device__ bool head_end(const Plan& plan) const { return vt == plan.vtiles - 1; }
  __device__ bool last(const Plan& plan) const { return head_end(plan) && head == last_head; }
  __device__ bool next(const Plan& plan, int nqk) {
    if (++vt < plan.vtiles) return true;
    vt = 0;
    ++head_no;
    if (++head <= last_head) return true;
    ++item_no;
    item += gridDim.x;
    return open(plan, nqk);
  }
};

// log2 of the weights of a token's sixteen columns from `col` on, where its block's tokens differ in hi.  Few
// blocks do: apart from the usual code, which does not fit the instruction cache as it is.
static __device__ __noinline__ void wide_exponents(const ChunkGates& G, int row, int col, float2 (&x)[8]) {
  const float hi = G.hi[row], lo = G.lo[row];
  for (int z = 0; z < 8; ++z)
    x[z] = make_float2((hi - G.hi[col + 2 * z]) + (lo - G.diag[col + 2 * z]),
                       (hi - G.hi[col + 2 * z + 1]) + (lo - G.diag[col + 2 * z + 1]));
}

template <int KP>
__global__ void __launch_bounds__(kThreads, 1)
    ssm_backward_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_dy,
                        const __grid_constant__ CUtensorMap map_h, const __grid_constant__ CUtensorMap map_g,
                        const __grid_constant__ CUtensorMap map_dq, const __grid_constant__ CUtensorMap map_dk,
                        const __grid_constant__ CUtensorMap map_dv, SsmBackwardProblem p, Plan plan, Workspace w,
                        bool tma) {
  using S = Smem<KP>;
  constexpr int PANELS = KP / 64;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t base = smem_u32(smem);
  BackwardGates* gates = reinterpret_cast<BackwardGates*>(smem + S::kGates);
  Sums& sums = *reinterpret_cast<Sums*>(smem + S::kSums);
  Bars& bar = *reinterpret_cast<Bars*>(smem + S::kBars);
  float (*wr)[16] = reinterpret_cast<float (*)[16]>(smem + S::kWr);  // w_r, 16 columns per group of warps
  volatile int* abort = &bar.abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const size_t plane = (size_t)p.K * p.V;
  if (tid == 0) {
    mbar_init(&bar.qk, 1), mbar_init(&bar.vd, 1), mbar_init(&bar.h, 1), mbar_init(&bar.g, 1);
    mbar_init(&bar.step_free, 16), mbar_init(&bar.vd_read, 16);
    mbar_init(&bar.scaled1, 16), mbar_init(&bar.scaled2, 16);
    mbar_init(&bar.s, 1), mbar_init(&bar.pds, 16), mbar_init(&bar.hd, 1), mbar_init(&bar.q_read, 16);
    mbar_init(&bar.gd, 1), mbar_init(&bar.done, 1), mbar_init(&bar.acc_free, 16);
    for (int i = 0; i < 2; ++i) mbar_init(&bar.gate[i], 1), mbar_init(&bar.gate_free[i], 17);
    mbar_init(&bar.sums, 16), mbar_init(&bar.sums_free, 1), mbar_init(&bar.out, 16), mbar_init(&bar.out_free, 1);
    bar.abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc(&bar.tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;
  bool ok = true;  // uniform in the warp
  auto wait = [&](uint64_t& b, int i) {
    if (ok) ok = warp_wait(&b, (uint32_t)i & 1u, abort);
    return ok;
  };
  Cursor at;
  bool more = at.start(plan, p.Nqk);

  if (warp < kWarpMma) {  // ------------------------------------------ element-wise
    const int quarter = warp & 3, group = warp >> 2, row = 32 * quarter + lane;
    const uint32_t t_lane = tmem + ((uint32_t)(32 * quarter) << 16);
    const uint32_t tv = base + S::kV, td = base + S::kDy;
    const int c0 = 16 * group;  // this warp's 16 of the 64 value columns
    bool sent_all = false;  // the step before sent dq and dk too
    for (int j = 0; more; ++j) {
      const int v0 = at.vt * VT, vw = min(VT, p.V - v0);
      if (j > 0) wait(bar.done, j - 1);         // (the scaled operand's place is read no more,
      if (sent_all) wait(bar.out_free, j - 1);  // nor does dk leave through it)
      wait(bar.gate[j & 1], j >> 1);
      if (!wait(bar.vd, j)) break;
      const ChunkGates& G = gates[j & 1].g;
      const float cum = G.hi[row] + G.lo[row], wk = G.wk[row];  // (hi counts between blocks alone)
      const float et = exp2_approx(cum + G.span[quarter][0]);
      const float wl = lane < 16 && c0 + lane < vw ? p.w_r[(size_t)at.head * p.V + v0 + c0 + lane] : 0.f;
      // exp(c) dy as an operand (and below w v, in the same place).
      auto put_scaled = [&](const uint4 (&from)[2], float f, uint64_t& ready) {
        const float2 f2 = make_float2(f, f);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t a = tile_at(0, row, 2 * group + c);
          float2 x[4];
          uint32_t o[4];
          unpack8(from[c], x);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 y = mul2(x[e], f2);
            o[e] = pack_bf16x2(y.x, y.y);
          }
          st_shared_v4(base + S::kScaled + a, make_uint4(o[0], o[1], o[2], o[3]));
        }
        fence_proxy_async_smem();
        warp_arrive(&ready, lane);
      };
      {
        const uint4 dr[2] = {ld_shared_v4(tile_at(td, row, 2 * group)),
                             ld_shared_v4(tile_at(td, row, 2 * group + 1))};
        put_scaled(dr, et, bar.scaled1);
      }

      // P and dS from S and dP, 16 columns at a time: pieces `group` and 7 - group of eight, so that
      // no warp of a quarter has both of the masked ones.
      if (j > 0 && !sent_all) wait(bar.out_free, j - 1);  // (the places of P and dS)
      if (at.vt == 0 && at.head_no > 0) wait(bar.sums_free, at.head_no - 1);
      if (!wait(bar.s, j)) break;
      tc_fence_after();
      {
        float rows = 0.f;
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          const int piece = x ? 7 - group : group, block = piece >> 1, ch = 2 * (piece & 3);
          const uint32_t tp = base + S::kP + (piece >> 2) * S::kTile, ts = base + S::kDs + (piece >> 2) * S::kTile;
          if (block > quarter) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              st_shared_v4(tile_at(tp, row, ch + c), make_uint4(0u, 0u, 0u, 0u));
              st_shared_v4(tile_at(ts, row, ch + c), make_uint4(0u, 0u, 0u, 0u));
            }
            continue;
          }
          float sc[16], dp[16];
          uint32_t po[8], so[8];
          float2 m[8];
          tmem_ld16_nowait(t_lane + kColS + 16 * piece, sc);
          tmem_ld16_nowait(t_lane + kColDp + 16 * piece, dp);
          int own = -1;  // the token's own column of these
          if (block < quarter) {
            const float u = exp2_approx(cum + G.span[quarter][block + 1]);
            const float2 u2 = make_float2(u, u);
            const float4* w4 = reinterpret_cast<const float4*>(G.wd + 16 * piece);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const float4 wv = w4[z];
              m[2 * z] = mul2(u2, make_float2(wv.x, wv.y));
              m[2 * z + 1] = mul2(u2, make_float2(wv.z, wv.w));
            }
          } else {  // a masked pair has decay 2^-infinity
            own = lane - 16 * (piece & 1);
            const float4* w4 = reinterpret_cast<const float4*>(G.diag + 16 * piece);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const float4 wv = w4[z];
              m[2 * z] = make_float2(cum - wv.x, cum - wv.y);
              m[2 * z + 1] = make_float2(cum - wv.z, cum - wv.w);
            }
            if (G.wide(quarter)) {
              tmem_ready(sc, dp);  // no load may be in flight across the call
              float2 x[8];
              wide_exponents(G, row, 16 * piece, x);
#pragma unroll
              for (int z = 0; z < 8; ++z) m[z] = x[z];
            }
#pragma unroll
            for (int z = 0; z < 8; ++z)
              m[z] = make_float2(exp2_approx(2 * z <= own ? m[z].x : -INFINITY),
                                 exp2_approx(2 * z + 1 <= own ? m[z].y : -INFINITY));
          }
          tmem_ready(sc, dp);
          // E (into sc) = P dP.
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int z = 0; z < 8; ++z) {
            const float2 d = make_float2(dp[2 * z], dp[2 * z + 1]);
            const float2 pv = mul2(make_float2(sc[2 * z], sc[2 * z + 1]), m[z]), sv = mul2(d, m[z]);
            float2 ev = mul2(pv, d);
            po[z] = pack_bf16x2(pv.x, pv.y);
            so[z] = pack_bf16x2(sv.x, sv.y);
            sum = add2(sum, ev);
            sc[2 * z] = ev.x, sc[2 * z + 1] = ev.y;
          }
          // Column sums over the warp's 32 rows: E through this piece's own place in the tiles of P
          // (columns 0 .. 7) and dS, read back four columns and four rows per lane, then across
          // eight lanes.
#pragma unroll
          for (int c = 0; c < 4; ++c)
            st_shared_v4(tile_at(c < 2 ? tp : ts, row, ch + (c & 1)),
                         make_uint4(__float_as_uint(sc[4 * c]), __float_as_uint(sc[4 * c + 1]),
                                    __float_as_uint(sc[4 * c + 2]), __float_as_uint(sc[4 * c + 3])));
          __syncwarp();
          const bool up = lane & 16, mid = lane & 8;
          // To the lanes without bit 2 of each column's four.
          auto to_columns = [&](float* to, float2 a01, float2 a23) {
            float k0 = up ? a23.x : a01.x, k1 = up ? a23.y : a01.y;
            k0 += __shfl_xor_sync(~0u, up ? a01.x : a23.x, 16);
            k1 += __shfl_xor_sync(~0u, up ? a01.y : a23.y, 16);
            float k = mid ? k1 : k0;
            k += __shfl_xor_sync(~0u, mid ? k0 : k1, 8);
            k += __shfl_xor_sync(~0u, k, 4);
            to += 16 * piece + 4 * (lane & 3) + (up ? 2 : 0) + (mid ? 1 : 0);
            if (!(lane & 4)) *to = at.vt ? *to + k : k;
          };
          float2 a01 = make_float2(0.f, 0.f), a23 = a01, b01 = a01, b23 = a01;
          const uint32_t from = lane & 2 ? ts : tp;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int u = (lane >> 2) + 8 * r;
            const uint4 q = ld_shared_v4(tile_at(from, 32 * quarter + u, ch + (lane & 1)));
            float2 e0 = make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
            float2 e1 = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
            a01 = add2(a01, e0);
            a23 = add2(a23, e1);
            if (block == quarter) {
              // In the rows' own block also, for column t and row u >= t, E over the piece's columns before
              // t (u's own left out): what passes t within the piece.  At the fourth lane the row's sum.
              const int n = u - 16 * (piece & 1) - 4 * (lane & 3);  // this lane's columns before u
              e0.x = n > 0 ? e0.x : 0.f, e0.y = n > 1 ? e0.y : 0.f;
              e1.x = n > 2 ? e1.x : 0.f, e1.y = n > 3 ? e1.y : 0.f;
              const float p2 = e0.x + e0.y, p3 = p2 + e1.x;
              float run = p3 + e1.y;
              float x = __shfl_up_sync(~0u, run, 1, 4);
              if (lane & 3) run += x;
              x = __shfl_up_sync(~0u, run, 2, 4);
              if (lane & 2) run += x;
              x = __shfl_up_sync(~0u, run, 1, 4);
              if ((lane & 3) == 0) x = 0.f;
              b01.x += n >= 0 ? x : 0.f, b01.y += n >= 1 ? x + e0.x : 0.f;
              b23.x += n >= 2 ? x + p2 : 0.f, b23.y += n >= 3 ? x + p3 : 0.f;
              if ((lane & 3) == 3 && !(piece & 1)) {
                float& to = sums.first[32 * quarter + u];
                to = at.vt ? to + run : run;
              }
            }
          }
          if (block == quarter) {
            to_columns(sums.own, a01, a23);
            to_columns(sums.col[quarter], b01, b23);
          } else {
            to_columns(sums.col[quarter], a01, a23);
            rows += sum.x + sum.y;
          }
          __syncwarp();
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            st_shared_v4(tile_at(tp, row, ch + c), make_uint4(po[4 * c], po[4 * c + 1], po[4 * c + 2], po[4 * c + 3]));
            st_shared_v4(tile_at(ts, row, ch + c), make_uint4(so[4 * c], so[4 * c + 1], so[4 * c + 2], so[4 * c + 3]));
          }
        }
        float& to = sums.row[group][row];
        to = at.vt ? to + rows : rows;
      }
      fence_proxy_async_smem();
      tc_fence_before();
      warp_arrive(&bar.pds, lane);

      // dw_r of the chunk: eight columns, four tokens per lane, by the quarters with the fewest scores.
      if (quarter < 2) {
        const int piece = 2 * group + quarter;
        float2 s[4] = {};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t a = tile_at(0, lane + 32 * r, piece);
          float2 x[4], y[4];
          unpack8(ld_shared_v4(tv + a), x);
          unpack8(ld_shared_v4(td + a), y);
#pragma unroll
          for (int e = 0; e < 4; ++e) s[e] = fma2(x[e], y[e], s[e]);
        }
        const bool up = lane & 16, mid = lane & 8, low = lane & 4;
        float2 h0 = up ? s[2] : s[0], h1 = up ? s[3] : s[1];
        const float2 g0 = up ? s[0] : s[2], g1 = up ? s[1] : s[3];
        h0.x += __shfl_xor_sync(~0u, g0.x, 16), h0.y += __shfl_xor_sync(~0u, g0.y, 16);
        h1.x += __shfl_xor_sync(~0u, g1.x, 16), h1.y += __shfl_xor_sync(~0u, g1.y, 16);
        float2 h = mid ? h1 : h0;
        const float2 g = mid ? h0 : h1;
        h.x += __shfl_xor_sync(~0u, g.x, 8), h.y += __shfl_xor_sync(~0u, g.y, 8);
        float k = (low ? h.y : h.x) + __shfl_xor_sync(~0u, low ? h.x : h.y, 4);
        k += __shfl_xor_sync(~0u, k, 2);
        k += __shfl_xor_sync(~0u, k, 1);
        const int col = 8 * piece + (up ? 4 : 0) + (mid ? 2 : 0) + (low ? 1 : 0);
        if ((lane & 3) == 0 && col < vw)
          w.par[((size_t)(at.b * plan.chunks + at.chunk) * p.N + at.head) * (2 + p.V) + 2 + v0 + col] = k;
      }

      // This token's v and dy, 16 columns: from here on their tiles are the products' alone.
      uint4 vr[2], dr[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        vr[c] = ld_shared_v4(tile_at(tv, row, 2 * group + c));
        dr[c] = ld_shared_v4(tile_at(td, row, 2 * group + c));
      }
      warp_arrive(&bar.vd_read, lane);

      // The state's part of the row sums: exp(c) (q H) . dy.
      if (!wait(bar.hd, j)) break;
      tc_fence_after();
      {
        float hi[16], lo[16];
        tmem_ld16_nowait(t_lane + kColS + c0, hi);
        tmem_ld16_nowait(t_lane + kColS + VT + c0, lo);
        float2 y[8];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float2 x[4];
          unpack8(dr[c], x);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[4 * c + e] = x[e];
        }
        tmem_ready(hi, lo);
        tc_fence_before();
        warp_arrive(&bar.q_read, lane);
        float2 dot = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          dot = fma2(add2(make_float2(hi[2 * e], hi[2 * e + 1]), make_float2(lo[2 * e], lo[2 * e + 1])), y[e], dot);
        float& to = sums.row_state[group][row];
        const float r = et * (dot.x + dot.y);
        to = at.vt ? to + r : r;
      }
      if (lane < 16) wr[group][lane] = wl;  // (every warp has read the step before's)
      put_scaled(vr, wk, bar.scaled2);

      // k G: its part of the column sums, and dv = P^T dy + w (k G) + w_r dy, which leaves through the
      // first half of P's tile.
      if (!wait(bar.gd, j)) break;
      tc_fence_after();
      float2 dot = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float hi[8], lo[8], a[8];
        tmem_ld8_nowait(t_lane + kColDp + c0 + 8 * c, hi);
        tmem_ld8_nowait(t_lane + kColDp + VT + c0 + 8 * c, lo);
        tmem_ld8_nowait(t_lane + kColS + c0 + 8 * c, a);
        float2 x[4], y[4];
        uint32_t o[4];
        unpack8(vr[c], x);
        unpack8(dr[c], y);
        tmem_ready(hi, lo, a);
        const float2 w2 = make_float2(wk, wk);
        const float4 w0 = reinterpret_cast<const float4*>(wr[group])[2 * c];
        const float4 w1 = reinterpret_cast<const float4*>(wr[group])[2 * c + 1];
        const float2 u[4] = {make_float2(w0.x, w0.y), make_float2(w0.z, w0.w), make_float2(w1.x, w1.y),
                             make_float2(w1.z, w1.w)};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 kg = mul2(w2, add2(make_float2(hi[2 * e], hi[2 * e + 1]), make_float2(lo[2 * e], lo[2 * e + 1])));
          dot = fma2(kg, x[e], dot);
          const float2 r = fma2(u[e], y[e], add2(make_float2(a[2 * e], a[2 * e + 1]), kg));
          o[e] = pack_bf16x2(r.x, r.y);
        }
        st_shared_v4(tile_at(base + S::kP, row, 2 * group + c), make_uint4(o[0], o[1], o[2], o[3]));
      }
      {
        float& to = sums.col_state[group][row];
        to = at.vt ? to + (dot.x + dot.y) : dot.x + dot.y;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar.step_free);
        mbar_arrive(&bar.gate_free[j & 1]);
        if (at.head_end(plan)) mbar_arrive(&bar.sums);
      }

      // dq, dk of the item: bf16 through dS's tile, and the other half of P's and the scaled
      // operand's; parts of a split item float32, a token per lane.
      sent_all = at.last(plan);
      if (sent_all) {
        if (!wait(bar.done, j)) break;
        tc_fence_after();
        constexpr int KC = KP / 4;  // columns per warp
#pragma unroll 1
        for (int c = 0; c < 2 * KC; c += 16) {
          const bool is_k = c >= KC;
          const int col = KC * group + (is_k ? c - KC : c);
          float a[16];
          tmem_ld16_nowait(t_lane + (is_k ? kColDk : kColDq) + col, a);
          tmem_ready(a);
          if (plan.splits > 1) {
            float* f = (is_k ? w.dkp : w.dqp) + ((size_t)at.item * KP + col) * L + row;
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e * L] = a[e];
          } else {
            const uint32_t to = is_k ? (col < 64 ? base + S::kP + S::kTile : base + S::kScaled)
                                     : base + S::kDs + (col >> 6) * S::kTile;
#pragma unroll
            for (int x = 0; x < 2; ++x)
              st_shared_v4(tile_at(to, row, ((col & 63) >> 3) + x),
                           make_uint4(pack_bf16x2(a[8 * x], a[8 * x + 1]), pack_bf16x2(a[8 * x + 2], a[8 * x + 3]),
                                      pack_bf16x2(a[8 * x + 4], a[8 * x + 5]), pack_bf16x2(a[8 * x + 6], a[8 * x + 7])));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.acc_free);
      }
      fence_proxy_async_smem();
      warp_arrive(&bar.out, lane);
      more = at.next(plan, p.Nqk);
    }
  } else if (warp == kWarpMma) {  // ---------------------------------- products
    const uint32_t id_ss = umma_idesc_bf16(128, 128, false);                   // both K-major
    const uint32_t id_st = umma_idesc_bf16_ab(128, 128, false, true);          // a state, high and low
    const uint32_t id_k = umma_idesc_bf16(128, KP, false);
    const uint32_t id_dq = umma_idesc_bf16_ab(128, KP, false, true), id_dk = umma_idesc_bf16_ab(128, KP, true, true);
    const uint32_t id_dv = umma_idesc_bf16_ab(128, VT, true, true);
    const uint32_t q = base + S::kQ, k = base + S::kK, v = base + S::kV, dy = base + S::kDy, st = base + S::kState;
    const uint32_t sc = base + S::kScaled, tp = base + S::kP, ts = base + S::kDs;
    constexpr int PANEL = L * 8 - 8;  // to the next panel of 64 columns, K-major
    const bool leader = lane == 0;
    for (int j = 0; more; ++j) {
      const bool first = at.first(plan);
      if (first) wait(bar.qk, at.item_no);
      if (j > 0) wait(bar.step_free, j - 1);
      if (!wait(bar.vd, j)) break;
      tc_fence_after();
      umma_steps<KP / 16, 2, 2, PANEL, PANEL>(leader, tmem + kColS, desc_k(q), desc_k(k), id_ss, false);
      umma_steps<4, 2, 2>(leader, tmem + kColDp, desc_k(dy), desc_k(v), id_ss, false);
      umma_commit_if(leader, &bar.s);
      if (first && at.item_no > 0) wait(bar.acc_free, at.item_no - 1);
      wait(bar.h, j);
      if (!wait(bar.scaled1, j)) break;
      tc_fence_after();
      umma_steps<4, 2, 2>(leader, tmem + kColDq, desc_k(sc), desc_k(st), id_k, !first);
      umma_steps<4, 2, 2>(leader, tmem + kColDq, desc_k(sc), desc_k(st + KP * VT * 2), id_k, true);
      if (!wait(bar.pds, j)) break;
      tc_fence_after();
      umma_steps<KP / 16, 2, 128, PANEL>(leader, tmem + kColS, desc_k(q), desc_mn(st, KP), id_st, false);
      umma_commit_if(leader, &bar.hd);
      umma_steps<L / 16, 2, 128, PANEL>(leader, tmem + kColDq, desc_k(ts), desc_mn(k, L), id_dq, true);
      umma_steps<L / 16, 128, 128>(leader, tmem + kColDk, desc_mn(ts, L), desc_mn(q, L), id_dk, !first);
      if (!wait(bar.q_read, j)) break;
      tc_fence_after();
      umma_steps<L / 16, 128, 128>(leader, tmem + kColS, desc_mn(tp, L), desc_mn(dy, L), id_dv, false);
      if (!wait(bar.g, j)) break;
      umma_steps<KP / 16, 2, 128, PANEL>(leader, tmem + kColDp, desc_k(k), desc_mn(st, KP), id_st, false);
      umma_commit_if(leader, &bar.gd);
      if (!wait(bar.scaled2, j)) break;
      tc_fence_after();
      umma_steps<4, 2, 2>(leader, tmem + kColDk, desc_k(sc), desc_k(st), id_k, true);
      umma_steps<4, 2, 2>(leader, tmem + kColDk, desc_k(sc), desc_k(st + KP * VT * 2), id_k, true);
      umma_commit_if(leader, &bar.done);
      more = at.next(plan, p.Nqk);
    }
  } else if (warp == kWarpLoad) {  // --------------------------------- loads
    for (int j = 0; more; ++j) {
      const int t0 = at.chunk * L, rows = min(L, p.T - t0), v0 = at.vt * VT, vw = min(VT, p.V - v0);
      const long long pair = (long long)at.b * p.N + at.head;
      if (at.first(plan)) {
        if (j > 0 && !wait(bar.done, j - 1)) break;
        if (tma) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&bar.qk, 2 * L * KP * 2);
#pragma unroll
            for (int x = 0; x < PANELS; ++x) {
              tma_load_4d(smem + S::kQ + panel(x, L), &map_q, &bar.qk, 64 * x, at.group, t0, at.b);
              tma_load_4d(smem + S::kK + panel(x, L), &map_k, &bar.qk, 64 * x, at.group, t0, at.b);
            }
          }
        } else {
          for (int x = 0; x < PANELS; ++x) {
            copy_tokens(base + S::kQ + panel(x, L),
                        p.q + at.b * p.sq.batch + t0 * p.sq.token + (long long)at.group * p.K + 64 * x, p.sq.token, rows, p.K - 64 * x, lane);
            copy_tokens(base + S::kK + panel(x, L),
                        p.k + at.b * p.sk.batch + t0 * p.sk.token + (long long)at.group * p.K + 64 * x, p.sk.token, rows, p.K - 64 * x, lane);
          }
          fence_proxy_async_smem();
          warp_arrive(&bar.qk, lane);
        }
      }
      if (j >= 2 && !wait(bar.gate_free[j & 1], (j >> 1) - 1)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bar.gate[j & 1], sizeof(BackwardGates));
        bulk_load(base + S::kGates + (j & 1) * (uint32_t)sizeof(BackwardGates), w.gates + pair * plan.chunks + at.chunk,
                  sizeof(BackwardGates), &bar.gate[j & 1]);
      }
      if (j > 0) wait(bar.vd_read, j - 1);
      if (j > 0 && !wait(bar.gd, j - 1)) break;
      if (tma) {
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar.vd, 2 * S::kTile);
          tma_load_4d(smem + S::kV, &map_v, &bar.vd, v0, at.head, t0, at.b);
          tma_load_4d(smem + S::kDy, &map_dy, &bar.vd, v0, at.head, t0, at.b);
        }
      } else {
        copy_tokens(base + S::kV, p.v + at.b * p.sv.batch + t0 * p.sv.token + (long long)at.head * p.V + v0, p.sv.token,
                    rows, vw, lane);
        copy_tokens(base + S::kDy, p.dy + (((size_t)at.b * p.T + t0) * p.N + at.head) * p.V + v0, (long long)p.N * p.V,
                    rows, vw, lane);
        fence_proxy_async_smem();
        warp_arrive(&bar.vd, lane);
      }
      // The next step's tiles on their way to L2: they are loaded late, when their places are free.
      if (tma && lane == 0) {
        Cursor to = at;
        if (to.next(plan, p.Nqk)) {
          const int pair_to = to.b * p.N + to.head;
          tma_prefetch_4d(&map_v, to.vt * VT, to.head, to.chunk * L, to.b);
          tma_prefetch_4d(&map_dy, to.vt * VT, to.head, to.chunk * L, to.b);
          for (int x = 0; x < 2; ++x) {
            tma_prefetch_4d(&map_h, to.vt * VT, 0, 2 * to.chunk + x, pair_to);
            tma_prefetch_4d(&map_g, to.vt * VT, 0, 2 * to.chunk + x, pair_to);
          }
          if (to.first(plan))
            for (int x = 0; x < PANELS; ++x) {
              tma_prefetch_4d(&map_q, 64 * x, to.group, to.chunk * L, to.b);
              tma_prefetch_4d(&map_k, 64 * x, to.group, to.chunk * L, to.b);
            }
        }
      }
      __syncwarp();
      // H once the products with the step before's G are done, G once those with H are.
#pragma unroll 1
      for (int s = 0; s < 2; ++s) {
        if (s == 0 && j > 0 && !wait(bar.done, j - 1)) break;
        if (s == 1 && !wait(bar.hd, j)) break;
        uint64_t* full = s ? &bar.g : &bar.h;
        if (tma) {
          if (lane == 0) {
            mbar_arrive_expect_tx(full, 2 * KP * VT * 2);
            for (int x = 0; x < 2; ++x)
              tma_load_4d(smem + S::kState + x * KP * VT * 2, s ? &map_g : &map_h, full, v0, 0, 2 * at.chunk + x, (int)pair);
          }
        } else {
          const uint16_t* src = s ? w.G + ((size_t)pair * plan.chunks + at.chunk) * 2 * plane
                                  : p.Hs + ((size_t)pair * (plan.chunks + 1) + at.chunk) * 2 * plane;
          copy_state<KP>(base + S::kState, src + v0, p.K, p.V, vw, lane);
          warp_arrive(full, lane);
        }
        __syncwarp();
      }
      if (!ok) break;
      more = at.next(plan, p.Nqk);
    }
    // Given up: whatever was started here arrives before the block ends (waits for what was not
    // started run out).
    if (!ok) {
      uint64_t* all[6] = {&bar.gate[0], &bar.gate[1], &bar.qk, &bar.vd, &bar.h, &bar.g};
      for (int s = 0; s < (tma ? 6 : 2); ++s)
        for (int phase = 0; phase < 2; ++phase) mbar_wait_bounded(all[s], phase, kWaitLimitCycles / 64);
    }
  } else if (warp == kWarpStore) {  // -------------------------------- stores
    for (int j = 0; more; ++j) {
      if (!wait(bar.out, j)) break;
      const int t0 = at.chunk * L, v0 = at.vt * VT;
      const bool both = at.last(plan) && plan.splits == 1;
      if (tma) {
        tma_store_4d_if(lane == 0, &map_dv, base + S::kP, v0, at.head, t0, at.b);
        if (both) {
#pragma unroll
          for (int x = 0; x < PANELS; ++x) {
            tma_store_4d_if(lane == 0, &map_dq, base + S::kDs + x * S::kTile, 64 * x, at.group, t0, at.b);
            tma_store_4d_if(lane == 0, &map_dk, x ? base + S::kScaled : base + S::kP + S::kTile, 64 * x, at.group, t0,
                            at.b);
          }
        }
        if (lane == 0) {
          bulk_commit_group();
          bulk_wait_group_read<0>();
        }
      } else {
        const int rows = min(L, p.T - t0);
        const size_t token = (size_t)at.b * p.T + t0;
        copy_out(p.dv + (token * p.N + at.head) * p.V + v0, base + S::kP, (long long)p.N * p.V, rows, min(VT, p.V - v0),
                 lane);
        for (int x = 0; x < PANELS && both; ++x) {
          const size_t to = (token * p.Nqk + at.group) * p.K + 64 * x;
          copy_out(p.dq + to, base + S::kDs + x * S::kTile, (long long)p.Nqk * p.K, rows, p.K - 64 * x, lane);
          copy_out(p.dk + to, x ? base + S::kScaled : base + S::kP + S::kTile, (long long)p.Nqk * p.K, rows, p.K - 64 * x,
                   lane);
        }
      }
      warp_arrive(&bar.out_free, lane);
      more = at.next(plan, p.Nqk);
    }
    if (lane == 0) bulk_wait_group<0>();
  } else {  // -------------------------------------------------------- the gate's gradient
    for (int j = 0; more; ++j) {
      if (!wait(bar.gate[j & 1], j >> 1)) break;
      if (at.head_end(plan)) {
        const long long pair = (long long)at.b * p.N + at.head;
        const BackwardGates& G = gates[j & 1];
        const float4 rho = reinterpret_cast<const float4*>(G.rho)[lane];
        const float4 asig = reinterpret_cast<const float4*>(G.asig)[lane], d = reinterpret_cast<const float4*>(G.d)[lane];
        const float* dots = w.dots + ((size_t)pair * plan.chunks + at.chunk) * plan.vtiles * 8;
        float across = lane < plan.vtiles * 8 ? dots[lane] * exp2_approx(G.g.total()) : 0.f;  // at most 16 parts
        if (!wait(bar.sums, at.head_no)) break;
        // Tokens 4 lane .. 4 lane + 3: r, l, da's own sum, and `pass`, E over all pairs that the token
        // separates: later one in a later block, by column (in the loop); both in its block's 16 columns, as
        // summed above; later one in its block, earlier one before these columns, by row.
        auto add = [](float4 a, const float* p, int lane) {
          const float4 b = reinterpret_cast<const float4*>(p)[lane];
          return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
        };
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        const int block = lane >> 3;  // of 32 tokens
        float4 r = zero, l = zero, full = add(zero, sums.own, lane), a = zero;
        float4 pass = add(zero, sums.col[block], lane);
        const float4 b = lane & 4 ? add(zero, sums.first, lane) : zero;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          r = add(r, sums.row_state[i], lane);
          l = add(l, sums.col_state[i], lane);
          a = add(a, sums.row[i], lane);
          const float4 c = i > block ? add(zero, sums.col[i], lane) : zero;
          const float c1 = c.x + c.y, c2 = c1 + c.z;
          float left = c2 + c.w;
#pragma unroll
          for (int s = 1; s < 32; s <<= 1) {
            const float x = __shfl_up_sync(~0u, left, s);
            if (lane >= s) left += x;
          }
          left = __shfl_up_sync(~0u, left, 1);
          if (i > block) {
            if (lane == 0) left = 0.f;
            full = make_float4(full.x + c.x, full.y + c.y, full.z + c.z, full.w + c.w);
            pass = make_float4(pass.x + left, pass.y + (left + c.x), pass.z + (left + c1), pass.w + (left + c2));
          }
        }
        warp_arrive(&bar.sums_free, lane);
        full = make_float4(full.x + l.x, full.y + l.y, full.z + l.z, full.w + l.w);
        {
          a.z += a.w, a.y += a.z, a.x += a.y;
          const float b2 = b.z + b.w, b1 = b.y + b2;
          float ra = a.x, rb = b.x + b1;  // over the block's lanes from this one on
#pragma unroll
          for (int s = 1; s < 8; s <<= 1) {
            const float x = __shfl_down_sync(~0u, ra, s, 8), y = __shfl_down_sync(~0u, rb, s, 8);
            if ((lane & 7) + s < 8) ra += x, rb += y;
          }
          ra = __shfl_down_sync(~0u, ra, 1, 8), rb = __shfl_down_sync(~0u, rb, 1, 8);
          if ((lane & 7) == 7) ra = rb = 0.f;
          if (!(lane & 4)) rb = 0.f;  // (tokens of the first 16 columns)
          const float rest = ra + rb;
          pass = make_float4(pass.x + (a.x + (b.x + b1) + rest), pass.y + (a.y + b1 + rest), pass.z + (a.z + b2 + rest),
                             pass.w + (a.w + b.w + rest));
        }
        // Sums of r over this token and the later ones, of l over the earlier ones.
        r.z += r.w, r.y += r.z, r.x += r.y;
        const float l1 = l.x + l.y, l2 = l1 + l.z;
        float after = r.x, before = l2 + l.w;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
          const float x = __shfl_down_sync(~0u, after, s), y = __shfl_up_sync(~0u, before, s);
          if (lane + s < 32) after += x;
          if (lane >= s) before += y;
          across += __shfl_xor_sync(~0u, across, s);
        }
        after = __shfl_down_sync(~0u, after, 1), before = __shfl_up_sync(~0u, before, 1);
        if (lane == 31) after = 0.f;
        if (lane == 0) before = 0.f;
        const float4 g = make_float4(across + (after + r.x) + before + pass.x, across + (after + r.y) + (before + l.x) + pass.y,
                                     across + (after + r.z) + (before + l1) + pass.z,
                                     across + (after + r.w) + (before + l2) + pass.w);
        const float4 da = make_float4(rho.x * full.x - asig.x * g.x, rho.y * full.y - asig.y * g.y,
                                      rho.z * full.z - asig.z * g.z, rho.w * full.w - asig.w * g.w);
        // (tokens past the sequence: d = 0, and every sum of theirs)
        float dalpha = -(d.x * g.x + d.y * g.y + d.z * g.z + d.w * g.w), dbeta = da.x + da.y + da.z + da.w;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          dalpha += __shfl_xor_sync(~0u, dalpha, o);
          dbeta += __shfl_xor_sync(~0u, dbeta, o);
        }
        if (lane == 0) {
          float* par = w.par + ((size_t)(at.b * plan.chunks + at.chunk) * p.N + at.head) * (2 + p.V);
          par[0] = dalpha, par[1] = dbeta;
        }
        const long long t = (long long)at.chunk * L + 4 * lane;
        uint16_t* to = p.da + ((size_t)at.b * p.T + t) * p.N + at.head;
        if (t < p.T) to[0] = f_to_bf16(da.x);
        if (t + 1 < p.T) to[p.N] = f_to_bf16(da.y);
        if (t + 2 < p.T) to[2 * (size_t)p.N] = f_to_bf16(da.z);
        if (t + 3 < p.T) to[3 * (size_t)p.N] = f_to_bf16(da.w);
      }
      warp_arrive(&bar.gate_free[j & 1], lane);
      more = at.next(plan, p.Nqk);
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

// Every chunk's gates: a warp per chunk of a (batch, head) pair.
__global__ void __launch_bounds__(128)
    ssm_gates_kernel(SsmBackwardProblem p, BackwardGates* __restrict__ out, long long pairs, int chunks) {
  const int lane = threadIdx.x & 31;
  const long long id = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (id >= pairs * chunks) return;
  const long long pair = id / chunks;
  const int n = (int)(pair % p.N);
  const uint16_t* ag = p.a + pair / p.N * p.sa.batch + n;
  const long long t0 = id % chunks * L + lane;
  const float alpha = p.alpha[n], beta = p.beta[n];
  float a[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) a[e] = t0 + 32 * e < p.T ? bf16_to_f(ag[(t0 + 32 * e) * p.sa.token]) : -INFINITY;
  BackwardGates& o = out[id];
  put_chunk_gates(
      o.g, [&](int e) { return e == 0 ? a[0] : e == 1 ? a[1] : e == 2 ? a[2] : a[3]; }, alpha, beta, lane);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float x = a[e] + beta, ex = expf(-fabsf(x));
    const float sig = x >= 0.f ? 1.f / (1.f + ex) : ex / (1.f + ex);
    o.rho[32 * e + lane] = sigmoid_over_softplus(x);
    o.asig[32 * e + lane] = alpha * sig;
    o.d[32 * e + lane] = ssm_gate(a[e], alpha, beta).x;
  }
}

// dq, dk: the splits' parts [item][column][token] added in order; a block per chunk of a batch row
// and q/k head and 32 columns, which turn through shared memory.
__global__ void __launch_bounds__(256)
    sum_splits_kernel(const float* __restrict__ dqp, const float* __restrict__ dkp, uint16_t* __restrict__ dq,
                      uint16_t* __restrict__ dk, Plan plan, int T, int Nqk, int K, int kp) {
  __shared__ float part[32][L + 1];
  const long long first = (long long)blockIdx.x * plan.splits;
  const int chunk = blockIdx.x % plan.chunks, group = blockIdx.x / plan.chunks % Nqk;
  const long long b = blockIdx.x / plan.chunks / Nqk;
  const float* src = blockIdx.y ? dkp : dqp;
  uint16_t* dst = (blockIdx.y ? dk : dq) + ((b * T + (long long)chunk * L) * Nqk + group) * K;
  const int rows = min(L, T - chunk * L);
  const int c0 = 32 * blockIdx.z;
  float4 s[4];  // 32 columns of 32 times four tokens, four of these per thread
#pragma unroll
  for (int e = 0; e < 4; ++e) s[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int i = 0; i < plan.splits; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = 8 * e + threadIdx.x / 32;
      const float4 x = reinterpret_cast<const float4*>(src + ((first + i) * kp + c0 + c) * L)[threadIdx.x % 32];
      s[e].x += x.x, s[e].y += x.y, s[e].z += x.z, s[e].w += x.w;
    }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float* to = &part[8 * e + threadIdx.x / 32][4 * (threadIdx.x % 32)];
    to[0] = s[e].x, to[1] = s[e].y, to[2] = s[e].z, to[3] = s[e].w;
  }
  __syncthreads();
  for (int id = threadIdx.x; id < 32 * L; id += 256) {
    const int r = id / 32, c = id % 32;
    if (r < rows && c0 + c < K) dst[(long long)r * Nqk * K + c0 + c] = f_to_bf16(part[c][r]);
  }
}

// Sums over the batch's chunks of the parts [rows][N][2 + V]: 32 columns by 32 slices of rows per
// block, the slices added in order.
__global__ void __launch_bounds__(1024)
    sum_params_kernel(const float* __restrict__ par, float* __restrict__ dalpha, float* __restrict__ dbeta,
                      float* __restrict__ dw_r, int rows, int N, int V) {
  __shared__ float part[32][33];
  const int width = N * (2 + V), c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (c < width)
    for (int r = threadIdx.y; r < rows; r += 32) s += par[(size_t)r * width + c];
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y || c >= width) return;
  s = 0.f;
  for (int i = 0; i < 32; ++i) s += part[i][threadIdx.x];
  const int n = c / (2 + V), j = c % (2 + V);
  if (j == 0)
    dalpha[n] = s;
  else if (j == 1)
    dbeta[n] = s;
  else
    dw_r[(size_t)n * V + j - 2] = s;
}

constexpr int kSms = 152;

// Splits of a group's heads: the fewest rounds of steps over the SMs, a split more only for a gain.
Plan make_plan(int B, int T, int N, int Nqk, int V) {
  Plan p;
  p.chunks = ssm_chunks(T);
  p.vtiles = (V + VT - 1) / VT;
  p.rep = N / Nqk;
  p.splits = 1;
  p.per_split = p.rep;
  const long long base = (long long)B * Nqk * p.chunks;
  double best = 1e30;
  for (int s = 1; s <= p.rep && s <= 16; ++s) {
    const int per = (p.rep + s - 1) / s, used = (p.rep + per - 1) / per;
    if (used != s) continue;
    const double cost = (double)((base * s + kSms - 1) / kSms) * (per + 0.5);
    if (cost < 0.97 * best) best = cost, p.splits = s, p.per_split = per;
  }
  p.items = base * p.splits;
  return p;
}

Workspace carve(float* ws, const Plan& plan, int B, int T, int N, int Nqk, int K, int V) {
  Workspace w;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += (n + 3) / 4 * 4;
    return ws ? ws + here : nullptr;
  };
  const size_t pairs = (size_t)B * N;
  w.G = reinterpret_cast<uint16_t*>(take(pairs * plan.chunks * K * V));
  w.segments = take(ssm_segment_floats(ssm_cut(B, T, N, V), B, N, K, V));
  w.dots = take(pairs * plan.chunks * plan.vtiles * 8);
  w.par = take((size_t)B * plan.chunks * N * (2 + V));
  w.gates = reinterpret_cast<BackwardGates*>(take(pairs * plan.chunks * (sizeof(BackwardGates) / 4)));
  const size_t part = plan.splits > 1 ? (size_t)plan.items * (K <= 64 ? 64 : 128) * L : 0;
  w.dqp = take(part);
  w.dkp = take(part);
  w.floats = at;
  return w;
}

template <int KP>
cudaError_t run(const SsmBackwardProblem& p, const Plan& plan, const Workspace& w, bool vec, cudaStream_t stream) {
  // At every launch: the attribute belongs to the current device.
  const cudaError_t attr =
      cudaFuncSetAttribute(ssm_backward_kernel<KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<KP>::kBytes);
  if (attr != cudaSuccess) return attr;
  const EncodeTiledFn enc = tensor_map_encoder();
  CUtensorMap mq{}, mk{}, mv{}, md{}, mh{}, mg{}, mdq{}, mdk{}, mdv{};
  const long long pairs = (long long)p.B * p.N;
  const Strides dense{(long long)p.T * p.N * p.V, (long long)p.N * p.V};
  const Strides dense_k{(long long)p.T * p.Nqk * p.K, (long long)p.Nqk * p.K};
  const bool tma = vec && enc && token_map(enc, &mq, p.q, p.K, p.Nqk, p.T, p.B, p.sq) &&
                   token_map(enc, &mk, p.k, p.K, p.Nqk, p.T, p.B, p.sk) &&
                   token_map(enc, &mv, p.v, p.V, p.N, p.T, p.B, p.sv) &&
                   token_map(enc, &md, p.dy, p.V, p.N, p.T, p.B, dense) &&
                   state_map(enc, &mh, p.Hs, p.K, p.V, 2LL * (plan.chunks + 1), pairs, KP) &&
                   state_map(enc, &mg, w.G, p.K, p.V, 2LL * plan.chunks, pairs, KP) &&
                   token_map(enc, &mdq, p.dq, p.K, p.Nqk, p.T, p.B, dense_k) &&
                   token_map(enc, &mdk, p.dk, p.K, p.Nqk, p.T, p.B, dense_k) &&
                   token_map(enc, &mdv, p.dv, p.V, p.N, p.T, p.B, dense);
  ssm_gates_kernel<<<(unsigned)((pairs * plan.chunks + 3) / 4), 128, 0, stream>>>(p, w.gates, pairs, plan.chunks);
  const unsigned blocks = (unsigned)(plan.items < kSms ? plan.items : kSms);
  ssm_backward_kernel<KP>
      <<<blocks, kThreads, Smem<KP>::kBytes, stream>>>(mq, mk, mv, md, mh, mg, mdq, mdk, mdv, p, plan, w, tma);
  return cudaGetLastError();
}

}  // namespace

size_t ssm_backward_workspace_bytes(int B, int T, int N, int Nqk, int K, int V) {
  return T > 0 ? sizeof(float) * carve(nullptr, make_plan(B, T, N, Nqk, V), B, T, N, Nqk, K, V).floats : 0;
}

cudaError_t launch_ssm_backward(const SsmBackwardProblem& p, cudaStream_t stream) {
  cudaError_t err = cudaSuccess;
  if (p.T == 0) {  // the final state is the first
    const size_t bytes = sizeof(float) * p.B * p.N * p.K * p.V;
    if (p.dH0 && p.dH_T && p.dH0 != p.dH_T)
      err = cudaMemcpyAsync(p.dH0, p.dH_T, bytes, cudaMemcpyDeviceToDevice, stream);
    else if (p.dH0 && !p.dH_T)
      err = cudaMemsetAsync(p.dH0, 0, bytes, stream);
    if (err == cudaSuccess) err = cudaMemsetAsync(p.dalpha, 0, sizeof(float) * p.N, stream);
    if (err == cudaSuccess) err = cudaMemsetAsync(p.dbeta, 0, sizeof(float) * p.N, stream);
    if (err == cudaSuccess) err = cudaMemsetAsync(p.dw_r, 0, sizeof(float) * p.N * p.V, stream);
    return err;
  }
  const Plan plan = make_plan(p.B, p.T, p.N, p.Nqk, p.V);
  if (plan.items > 0x7fffffffLL) return cudaErrorInvalidValue;  // (thousands of gigabytes of k and v)
  const Workspace w = carve(p.ws, plan, p.B, p.T, p.N, p.Nqk, p.K, p.V);
  const Strides dense{(long long)p.T * p.N * p.V, (long long)p.N * p.V};
  const bool vec = rows_of_16(p.q, p.sq, p.K) && rows_of_16(p.k, p.sk, p.K) && rows_of_16(p.v, p.sv, p.V) &&
                   rows_of_16(p.dy, dense, p.V) && aligned_to(p.dq, 16) && aligned_to(p.dk, 16) &&
                   aligned_to(p.dv, 16);
  StateProblem s{p.q, p.dy, p.a, p.alpha, p.beta, p.sq, dense, p.sa, p.B, p.T, p.N, p.Nqk, p.K, p.V, p.dH_T};
  s.status = p.status;
  const SsmCut cut = ssm_cut(p.B, p.T, p.N, p.V);
  if (cut.segments > 1) {
    err = launch_ssm_segments(s, cut, true, vec, w.segments, stream);
    if (err != cudaSuccess) return err;
    s.from_state = w.segments;
  }
  s.to = p.dH0, s.kept = w.G, s.Hs = p.Hs, s.dots = w.dots;
  err = launch_ssm_kept_states(s, cut, true, vec, stream);
  if (err != cudaSuccess) return err;
  err = p.K <= 64 ? run<64>(p, plan, w, vec, stream) : run<128>(p, plan, w, vec, stream);
  if (err != cudaSuccess) return err;
  if (plan.splits > 1)
    sum_splits_kernel<<<dim3((unsigned)(plan.items / plan.splits), 2, (p.K + 31) / 32), 256, 0, stream>>>(
        w.dqp, w.dkp, p.dq, p.dk, plan, p.T, p.Nqk, p.K, p.K <= 64 ? 64 : 128);
  const int width = p.N * (2 + p.V);
  sum_params_kernel<<<(width + 31) / 32, dim3(32, 32), 0, stream>>>(w.par, p.dalpha, p.dbeta, p.dw_r, p.B * plan.chunks,
                                                                   p.N, p.V);
  return cudaGetLastError();
}

}  // namespace m2rnn
