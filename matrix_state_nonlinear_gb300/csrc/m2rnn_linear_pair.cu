// m2rnn_linear_pair.cu — the 8-bit projection of many tokens: tiles of 256 tokens by 256 channels on pairs
// of SMs.
//
// Bound by the tensor cores.  A pair (a cluster of two blocks) shares each tile's operands: every block loads
// 128 rows of tokens and 128 of weights a stage and the product, issued by the first block, reads both
// blocks' shared memory, so that a stage's 32 KB feed 512 cycles of an SM's tensor core (a 128 x 256 tile
// of one SM would load 48).  Block r's accumulators hold tokens 128 r .. of the tile, a token per lane, all 256
// channels, and leave by 32-byte stores, a whole sector each.  Blocks stay on their SM and take tiles
// in turn; the next tile's products run while the last one's results leave.  Two buffers of 256 columns and
// the scales would need 536 columns of tensor memory, so the buffers overlap in 32 columns, which are read
// first: the next tile starts as soon as these are out.
// Measured, 16384 x 4096 x 8192: 307 us (3.6 PFLOP/s; the tensor cores work in 87 % of the cycles, at the clock
// that the power allows), 362 us in a long run at the power limit; 8192 x 2048 x 4384: 50 us.
#include "m2rnn_fp8_tc.cuh"

namespace m2rnn {
namespace {

constexpr int kRows = 128;                // rows of each operand per block and stage
constexpr int kTile = 2 * kRows;          // tokens and channels of a tile
constexpr int kStages = 6;
constexpr int kOperand = kRows * kBlockK, kStage = 2 * kOperand;
constexpr int kScaleStages = 3, kScaleWord = 512 + 1024, kScaleStage = 4 * kScaleWord;  // 128 tokens, 256 channels
constexpr int kScales = kStages * kStage;
constexpr int kTurn = kScales + kScaleStages * kScaleStage;  // 32 tokens by 32 channels of two bytes for each epilogue warp
constexpr int kTurnBytes = 32 * (32 * 2 + 4);
constexpr int kSmemBytes = kTurn + 4 * kTurnBytes + 1024;    // 1024: to align the first stage
constexpr int kEpilogueWarps = 4, kWarpLoad = 4, kWarpMma = 5, kWarpScale = 6, kThreads = 224;
constexpr int kTmemCols = 512, kColSecond = 224, kColScale = 480;  // scales: two sets of 4 + 8 columns
constexpr int kRun = 8;                   // token tiles that share a run of channel tiles

struct Bars {
  uint64_t full[kStages], empty[kStages], scale_full[kScaleStages], scale_empty[kScaleStages], done[2], early;
  uint32_t tmem;
  int abort;
};

// The barrier of both blocks completes when everything issued so far is done.
__device__ __forceinline__ void commit_pair_if(bool pred, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3), "r"((int)pred)
      : "memory");
}
// A load whose bytes count on a barrier (cluster address) that may be the other block's.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

// A whole warp waits for arrivals that may come from the other block.
__device__ __forceinline__ bool pair_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(~0u, mbar_wait_cluster(bar, parity, kWaitLimitCycles, abort));
}

// Tile t of the raster: runs of kRun token tiles by all channel tiles, so that the tiles in flight share
// their operands in L2.
__device__ __forceinline__ int2 tile_at_index(int t, int token_tiles, int channel_tiles) {
  const int run = t / (kRun * channel_tiles), first = run * kRun, wide = min(kRun, token_tiles - first);
  const int in = t - run * kRun * channel_tiles;
  return make_int2(first + in % wide, in / wide);
}

// One block to an SM, said to the compiler: left alone it keeps to 128 registers and spills (8192 x 4096 x 8192: 181
// us instead of 172).
template <typename Out>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                       LinearProblem p, int token_tiles, int channel_tiles, bool vec) {
  extern __shared__ unsigned char raw[];
  __shared__ Bars bar;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int blocks = scale_blocks(p.K), tiles = token_tiles * channel_tiles;
  volatile int* abort = &bar.abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&bar.full[s], 1), mbar_init(&bar.empty[s], 1);
    for (int s = 0; s < kScaleStages; ++s) mbar_init(&bar.scale_full[s], 2), mbar_init(&bar.scale_empty[s], 1);
    mbar_init(&bar.done[0], 1), mbar_init(&bar.done[1], 1);
    mbar_init(&bar.early, 2 * kEpilogueWarps);
    bar.abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bar.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  wait_for_launch_before();
  cluster_sync_all();  // the other block's barriers are ready
  tc_fence_after();
  const uint32_t tmem = bar.tmem;
  bool ok = true;
  // Steps are counted over all tiles: step g is stage g % kStages, its turn g / kStages.
  auto free_stage = [&](int g) {
    if (g >= kStages) ok = warp_wait(&bar.empty[g % kStages], (uint32_t)(g / kStages - 1) & 1u, abort);
    return ok;
  };

  if (warp == kWarpLoad) {
    int g = 0;
    for (int t = pair; t < tiles && ok; t += pairs) {
      const int2 at = tile_at_index(t, token_tiles, channel_tiles);
      for (int i = 0; i < blocks && free_stage(g); ++i, ++g) {
        if (lane == 0) {
          const int s = g % kStages;
          const uint32_t to = base + s * kStage, full = mapa_shared(smem_u32(&bar.full[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&bar.full[s], 2 * kStage);
          tma_load_2d_pair(to, &map_x, full, i * kBlockK, at.x * kTile + rank * kRows);
          tma_load_2d_pair(to + kOperand, &map_w, full, i * kBlockK, at.y * kTile + rank * kRows);
        }
        __syncwarp();
      }
    }
  } else if (warp == kWarpScale) {
    // Groups are counted over all tiles as the steps are: group h is slot h % kScaleStages.
    ScaleWords<4> x;
    ScaleWords<2> w;
    x.blocks = w.blocks = blocks;
    x.words = blocks % kQuad == 0 && reinterpret_cast<uintptr_t>(p.x_scales) % kQuad == 0;
    w.words = blocks % kQuad == 0 && reinterpret_cast<uintptr_t>(p.w_scales) % kQuad == 0;
    auto aim = [&](int t) {
      const int2 at = tile_at_index(t, token_tiles, channel_tiles);
#pragma unroll
      for (int c = 0; c < 4; ++c) x.aim(c, p.x_scales, (long long)at.x * kTile + rank * kRows + 32 * c + lane, p.M);
#pragma unroll
      for (int c = 0; c < 2; ++c) w.aim(c, p.w_scales, at.y * 2 + c, scale_blocks(p.N));
      x.fetch(0), w.fetch(0);
    };
    if (pair < tiles) aim(pair);
    int h = 0;
    for (int t = pair; t < tiles && ok; t += pairs) {
      for (int i = 0; i < blocks; i += kGroup, ++h) {
        uint32_t u[4][4], v[2][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
          for (int r = 0; r < 4; ++r) u[q][r] = x.word(r, q, i);
          v[0][q] = w.word(0, q, i), v[1][q] = w.word(1, q, i);
        }
        if (i + kGroup < blocks)
          x.fetch(i + kGroup), w.fetch(i + kGroup);
        else if (t + pairs < tiles)
          aim(t + pairs);
        const int s = h % kScaleStages;
        if (h >= kScaleStages && !(ok = warp_wait(&bar.scale_empty[s], (uint32_t)(h / kScaleStages - 1) & 1u, abort)))
          break;
        const uint32_t to = base + kScales + s * kScaleStage + lane * 16;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          st_shared_v4(to + q * kScaleWord, make_uint4(u[q][0], u[q][1], u[q][2], u[q][3]));
          st_shared_v4(to + q * kScaleWord + 512, make_uint4(v[0][q], v[0][q], v[0][q], v[0][q]));
          st_shared_v4(to + q * kScaleWord + 1024, make_uint4(v[1][q], v[1][q], v[1][q], v[1][q]));
        }
        // A release that other blocks see takes some 1800 cycles: once in 16 stages that passes unnoticed.
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&bar.scale_full[s]), 0));
      }
    }
  } else if (warp == kWarpMma) {
    // Stage s and scale slot hs, with the parities of their turns.
    const bool leader = elect_one_sync();
    int s = 0, hs = 0, n = 0;
    uint32_t turn = 0, scale_turn = 0, scales = 0;
    for (int t = pair; rank == 0 && t < tiles && ok; t += pairs, ++n) {
      if (n > 0 && !(ok = warp_wait(&bar.early, (uint32_t)(n - 1) & 1u, abort))) break;
      tc_fence_after();
      const uint32_t d = tmem + (n & 1 ? kColSecond : 0);
      for (int i0 = 0; i0 < blocks && ok; i0 += kQuad) {
        if (i0 % kGroup == 0) {
          if (!(ok = pair_wait(&bar.scale_full[hs], scale_turn, abort))) break;
          tc_fence_after();
          scales = base + kScales + hs * kScaleStage;
        }
        const uint32_t sa = tmem + kColScale + 12 * (i0 / kQuad & 1);
        copy_scales_if<true>(leader, sa, scales);
        copy_scales_if<true>(leader, sa + 4, scales + 512);
        copy_scales_if<true>(leader, sa + 8, scales + 1024);
        scales += kScaleWord;
        if (i0 % kGroup == kGroup - kQuad || i0 + kQuad >= blocks) {
          commit_pair_if(leader, &bar.scale_empty[hs]);
          if (++hs == kScaleStages) hs = 0, scale_turn ^= 1;
        }
#pragma unroll
        for (int j = 0; j < kQuad; ++j) {
          if (i0 + j >= blocks || !(ok = issue_wait(&bar.full[s], turn, abort))) break;
          tc_fence_after();
          const uint32_t at = base + s * kStage;
          umma4_fp8_if<true>(leader, d, desc_k(at), desc_k(at + kOperand), idesc_fp8(kTile, kTile, j), sa, sa + 4,
                             i0 + j > 0);
          commit_pair_if(leader, &bar.empty[s]);
          if (++s == kStages) s = 0, turn ^= 1;
        }
      }
      if (ok) commit_pair_if(leader, &bar.done[n & 1]);
    }
  } else {
    int n = 0;
    for (int t = pair; t < tiles; t += pairs, ++n) {
      const int2 at = tile_at_index(t, token_tiles, channel_tiles);
      if (!(ok = warp_wait(&bar.done[n & 1], (uint32_t)(n >> 1) & 1u, abort))) break;
      tc_fence_after();
      const long long m = (long long)at.x * kTile + rank * kRows + 32 * warp + lane;
      const uint32_t from = tmem + ((uint32_t)(32 * warp) << 16) + (n & 1 ? kColSecond : 0);
      Out* out = static_cast<Out*>(p.out) + m * p.N;
#pragma unroll 1
      for (int j = 0; j < kTile / 32; ++j) {
        const int c = n & 1 ? j : (j + kTile / 32 - 1) % (kTile / 32);  // the columns that both buffers have first
        float v[32];
        tmem_ld16_nowait(from + 32 * c, v);
        tmem_ld16_nowait(from + 32 * c + 16, v + 16);
        tmem_ready(v);
        if (j == 0) {
          tc_fence_before();
          __syncwarp();
          // Nothing but these loads, which are complete, has to come before: a release that other blocks see would
          // wait for the last tile's stores.
          if (lane == 0)
            asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(smem_u32(&bar.early), 0))
                         : "memory");
        }
        const int n0 = at.y * kTile + 32 * c;
        if (vec && m < p.M) {
          constexpr int V = 32 / sizeof(Out);
#pragma unroll
          for (int k = 0; k < 32; k += V) {
            uint32_t u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if constexpr (sizeof(Out) == 4)
                u[e] = __float_as_uint(v[k + e]);
              else
                u[e] = pack_bf16x2(v[k + 2 * e], v[k + 2 * e + 1]);
            }
            if (n0 + k < p.N)
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out + n0 + k), "r"(u[0]),
                           "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                           : "memory");
          }
        }
        if (!vec) {
          // Rows that do not start on whole sectors: turned in shared memory, so that a warp writes neighbouring
          // channels of one token (of 32-bit results 16 tokens after the other 16, for want of room).
          constexpr int kTokens = 64 / sizeof(Out), kRow = 32 * sizeof(Out) + 4;  // 4: rows in different banks
          static_assert(kTokens * kRow <= kTurnBytes, "room");
          const uint32_t turn = base + kTurn + warp * kTurnBytes;
#pragma unroll
          for (int part = 0; part < 32 / kTokens; ++part) {
            __syncwarp();
            if (lane / kTokens == part)
#pragma unroll
              for (int k = 0; k < 8 * (int)sizeof(Out); ++k) {
                uint32_t u;
                if constexpr (sizeof(Out) == 4)
                  u = __float_as_uint(v[k]);
                else
                  u = pack_bf16x2(v[2 * k], v[2 * k + 1]);
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(turn + lane % kTokens * kRow + 4 * k), "r"(u) : "memory");
              }
            __syncwarp();
            const long long first = m - lane + part * kTokens;
            const int live = n0 + lane < p.N ? (int)max(0LL, min((long long)kTokens, p.M - first)) : 0;
            Out* to = static_cast<Out*>(p.out) + first * p.N + n0 + lane;
#pragma unroll 8
            for (int t = 0; t < kTokens; ++t, to += p.N) {
              uint32_t u;
              asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u) : "r"((turn + t * kRow + lane * (int)sizeof(Out)) & ~3u));
              if (t < live) {
                if constexpr (sizeof(Out) == 4)
                  *to = __uint_as_float(u);
                else
                  *to = (uint16_t)(lane & 1 ? u >> 16 : u);
              }
            }
          }
        }
        __syncwarp();  // loads from tensor memory are the whole warp's
      }
    }
  }
  if (!ok && lane == 0) {
    *abort = 1;
    atomicExch(p.status, kStatusTimeout);
  }
  // Given up: loads that were started, by either block, arrive before the pair ends.
  if (!ok && warp == kWarpLoad && rank == 0)
    for (int phase = 0; phase < 2; ++phase)
      for (int s = 0; s < kStages; ++s) mbar_wait_bounded(&bar.full[s], phase, kWaitLimitCycles / 64);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // nothing of the other block reaches this one any more
  if (warp == kWarpMma)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

template <typename Out>
cudaError_t run(const LinearProblem& p, cudaStream_t stream) {
  // At every launch: the attribute belongs to the current device.
  const cudaError_t attr =
      cudaFuncSetAttribute(linear_pair_kernel<Out>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (attr != cudaSuccess) return attr;
  const EncodeTiledFn enc = tensor_map_encoder();
  CUtensorMap mw{}, mx{};
  if (!enc || !byte_map(enc, &mw, p.w, p.K, p.N, p.w_row, kRows) || !byte_map(enc, &mx, p.x, p.K, p.M, p.x_row, kRows))
    return cudaErrorNotSupported;
  const int tokens = (p.M + kTile - 1) / kTile, channels = (p.N + kTile - 1) / kTile;
  const long long tiles = (long long)tokens * channels;
  const bool vec = p.N % (32 / (int)sizeof(Out)) == 0 && aligned_to(p.out, 32);
  const unsigned pairs = (unsigned)(tiles < 76 ? tiles : 76);
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(2 * pairs);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = kSmemBytes;
  c.stream = stream;
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &a;
  c.numAttrs = p.follows ? 1 : 0;
  return cudaLaunchKernelEx(&c, linear_pair_kernel<Out>, mx, mw, p, tokens, channels, vec);
}

}  // namespace

cudaError_t launch_linear_pair(const LinearProblem& p, cudaStream_t stream) {
  return p.out_f32 ? run<float>(p, stream) : run<uint16_t>(p, stream);
}

}  // namespace m2rnn
