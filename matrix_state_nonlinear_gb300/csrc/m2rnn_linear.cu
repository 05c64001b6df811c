// m2rnn_linear.cu — product of 8-bit activations and weights with block scales.
//
//   out[m, n] = sum_k x[m, k] sx[m, k / 128] w[n, k] sw[n / 128, k / 128]
//
// The scales are powers of two, so the tensor cores apply them exactly (kind::mxf8f6f4) and the sum over
// all of K stays in one float32 accumulator in tensor memory.
//
// This kernel takes few and middling numbers of tokens and is bound by the weights' way from memory, and
// below a few megabytes by latency.  A block takes 128 channels (the product's rows, so that the weights fill
// the tensor core however few tokens there are) by NT tokens.  Where that gives fewer blocks than SMs, a
// cluster of up to 8 blocks shares a tile, each with a stretch of K.  Every block then writes each of the
// others' share of the tokens into that block's shared memory and adds up its own share in the order of K: one
// barrier of the cluster, nothing read from afar (half a microsecond less).  Up to 16 tokens of bf16 are
// quantised on the way in, by the warps that later write the results and four more (64 tokens would take 26 us
// that way, 13 with a launch before, 4096 x 8192: every block reads all rows).
// Measured, weights from memory: 64 x 4096 x 8192: 11.3 us (3.1 TB/s of weights and tokens), 11.7 with the quantising;
// 16 x 2048 x 4384: 6.8 us with it (5.3 alone with the weights in L2).
#include "m2rnn_fp8_tc.cuh"

namespace m2rnn {
namespace {

constexpr int MT = 128;  // channels of a tile
constexpr int kEpilogueWarps = 4, kWarpLoad = 4, kWarpMma = 5, kWarpScale = 6, kWarps = 7;
constexpr int kQuantWarps = 8;  // the epilogue's four and four more, behind the others
template <bool RAW>
constexpr int kThreads = 32 * (RAW ? kWarps + kQuantWarps - kEpilogueWarps : kWarps);

template <int NT, bool SPLIT>
struct Smem {
  static constexpr int kStages = NT <= 32 ? 8 : NT == 64 ? 7 : 6;
  static constexpr int kA = MT * kBlockK, kB = NT * kBlockK, kStage = kA + kB;
  static constexpr int kScaleStages = 4, kScaleStage = 1024;  // words of the channels and the tokens
  static constexpr int kScales = kStages * kStage;
  // The tile's parts that this block sums: [blocks of the cluster][its share of the tokens][channels] floats.  Those
  // of a block alone, or of 128 tokens, which would leave room for four stages, lie where the stages were; then
  // the cluster's blocks meet before they write there.
  static constexpr bool kOver = !SPLIT || NT == 128;
  static constexpr int kEnd = kScales + kScaleStages * kScaleStage, kParts = kOver ? 0 : kEnd;
  static constexpr int kBytes = kEnd + (kOver ? 0 : (NT + 7) * MT * 4) + 1024;  // 1024: to align the first stage
  static constexpr int kColScale = NT;                                   // two sets of 4 + 4 columns
  static constexpr int kTmemCols = NT <= 16 ? 32 : NT <= 32 ? 64 : NT <= 64 ? 128 : 256;
};
template <int S, int Q>
struct Bars {
  uint64_t full[S], empty[S], scale_full[Q], scale_empty[Q], done;
  uint32_t tmem;
  int abort;
};

// Eight bf16 values of a row from k on, zeros behind its K values.  The general case stays out of line: the
// loop it would be unrolled into does not fit the instruction cache.
__device__ __noinline__ uint4 load_any(const uint16_t* row, int k, int K) {
  uint32_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = k + i < K ? row[k + i] : 0u;
  return make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
}

template <int NT, bool RAW, bool SPLIT, typename Out>
__global__ void __launch_bounds__(kThreads<RAW>)
    linear_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, LinearProblem p,
                  int token_tiles, int split_, bool raw_vec, bool vec) {
  using S = Smem<NT, SPLIT>;
  constexpr int ST = S::kStages, SQ = S::kScaleStages;
  extern __shared__ unsigned char raw[];
  __shared__ Bars<ST, SQ> bar;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = SPLIT ? split_ : 1;
  const int tile = blockIdx.x / split, rank = blockIdx.x % split;  // a cluster is a tile's blocks
  const int n0 = tile / token_tiles * MT, m0 = tile % token_tiles * NT;
  // Stretches of K are of whole words of scales.
  const int all = scale_blocks(p.K), quads = (all + kQuad - 1) / kQuad;
  const int begin = kQuad * (int)((long long)quads * rank / split),
            end = min(all, kQuad * (int)((long long)quads * (rank + 1) / split));
  volatile int* abort = &bar.abort;

  const int steps = end - begin;
  // Step g is stage g % ST, its turn g / ST; its scales are byte g % 4 of word g / 4.
  auto load_w = [&](int g) {
    const int s = g % ST;
    mbar_arrive_expect_tx(&bar.full[s], RAW ? S::kA : S::kStage);
    tma_load_2d(base + s * S::kStage, &map_w, &bar.full[s], (begin + g) * kBlockK, n0);
  };
  auto load_x = [&](int g) {
    const int s = g % ST;
    if (!RAW) tma_load_2d(base + s * S::kStage + S::kA, &map_x, &bar.full[s], (begin + g) * kBlockK, m0);
  };
  // The first loads leave before anything else, those of the weights before the launch that writes x is over.
  if (warp == kWarpLoad && lane == 0) {
    for (int s = 0; s < ST; ++s) mbar_init(&bar.full[s], 1), mbar_init(&bar.empty[s], 1);
    for (int s = 0; s < SQ; ++s)
      mbar_init(&bar.scale_full[s], RAW ? 1 + kQuantWarps : 1), mbar_init(&bar.scale_empty[s], 1);
    mbar_init(&bar.done, 1);
    bar.abort = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    for (int g = 0; g < min(ST, steps); ++g) load_w(g);
    wait_for_launch_before();
    for (int g = 0; g < min(ST, steps); ++g) load_x(g);
  }
  if (warp == kWarpMma) tmem_alloc(&bar.tmem, S::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;
  constexpr bool kMeet = SPLIT && S::kOver;
  if (SPLIT && !kMeet) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this block has started
  bool ok = true;
  auto stage_free = [&](int g) {
    if (g >= ST) ok = warp_wait(&bar.empty[g % ST], (uint32_t)(g / ST - 1) & 1u, abort);
    return ok;
  };
  auto scales_free = [&](int h) {
    if (h >= SQ) ok = warp_wait(&bar.scale_empty[h % SQ], (uint32_t)(h / SQ - 1) & 1u, abort);
    return ok;
  };

  if (warp == kWarpLoad) {
    for (int g = ST; g < steps && stage_free(g); ++g) {
      if (lane == 0) load_w(g), load_x(g);
      __syncwarp();
    }
  } else if (warp == kWarpScale) {
    constexpr int R = (NT + 31) / 32;
    ScaleWords<1> w;
    ScaleWords<R> x;
    w.blocks = x.blocks = all;
    const bool words = all % kQuad == 0;
    w.words = words && reinterpret_cast<uintptr_t>(p.w_scales) % kQuad == 0;
    x.words = words && reinterpret_cast<uintptr_t>(p.x_scales) % kQuad == 0;
    w.aim(0, p.w_scales, n0 / kScaleBlock, scale_blocks(p.N));
#pragma unroll
    for (int c = 0; c < R; ++c) x.aim(c, p.x_scales, m0 + 32 * c + lane, RAW ? 0 : p.M);
    w.fetch(begin);
    wait_for_launch_before();
    x.fetch(begin);
    for (int i = begin, h = 0; i < end && ok; i += kGroup) {
      uint32_t v[4], u[4][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[q] = w.word(0, q, i);
#pragma unroll
        for (int r = 0; r < 4; ++r) u[q][r] = x.word(r < R ? r : 0, q, i);
      }
      if (i + kGroup < end) w.fetch(i + kGroup), x.fetch(i + kGroup);
#pragma unroll
      for (int q = 0; q < 4; ++q, ++h) {
        if (i + q * kQuad >= end || !scales_free(h)) break;
        const uint32_t to = base + S::kScales + h % SQ * S::kScaleStage + lane * 16;
        st_shared_v4(to, make_uint4(v[q], v[q], v[q], v[q]));
        if (!RAW) st_shared_v4(to + 512, make_uint4(u[q][0], u[q][1], u[q][2], u[q][3]));
        fence_proxy_async_smem();
        warp_arrive(&bar.scale_full[h % SQ], lane);
      }
    }
  } else if (warp == kWarpMma) {
    const bool leader = elect_one_sync();
    int s = 0, hs = 0;
    uint32_t turn = 0, scale_turn = 0;
    for (int i0 = begin; i0 < end && ok; i0 += kQuad) {
      if (!(ok = issue_wait(&bar.scale_full[hs], scale_turn, abort))) break;
      tc_fence_after();
      const uint32_t sa = tmem + S::kColScale + 8 * (hs & 1), scales = base + S::kScales + hs * S::kScaleStage;
      copy_scales_if<false>(leader, sa, scales);
      copy_scales_if<false>(leader, sa + 4, scales + 512);
      umma_commit_if(leader, &bar.scale_empty[hs]);
      if (++hs == SQ) hs = 0, scale_turn ^= 1;
#pragma unroll
      for (int j = 0; j < kQuad; ++j) {
        if (i0 + j >= end || !(ok = issue_wait(&bar.full[s], turn, abort))) break;
        tc_fence_after();
        const uint32_t at = base + s * S::kStage;
        umma4_fp8_if<false>(leader, tmem, desc_k(at), desc_k(at + S::kA), idesc_fp8(MT, NT, j), sa, sa + 4,
                            i0 + j > begin);
        umma_commit_if(leader, &bar.empty[s]);
        if (++s == ST) s = 0, turn ^= 1;
      }
    }
    if (ok) umma_commit_if(leader, &bar.done);
  } else {  // --------------- RAW: eight warps quantise
    if constexpr (RAW) {
      // 16 threads take 128 values of a row, eight each.  A word's four steps are handed over at once, with their
      // scales; as each is done, the one four steps on starts on its way.
      static_assert(NT == 16 && kQuantWarps == 8, "a row for every 16 threads");
      const int id = warp < kEpilogueWarps ? threadIdx.x : threadIdx.x - 32 * (kWarps - kEpilogueWarps);
      const int r = id >> 4, piece = id & 15;
      const bool live = m0 + r < p.M;  // products of rows that are not there go nowhere
      const uint16_t* row = p.raw + (live ? (m0 + r) * p.x_row : 0);
      uint4 word[kQuad];
      auto fetch = [&](int g) {
        const int k = (begin + g) * kBlockK + piece * 8;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (raw_vec && live && g < steps && k < p.K) u = *reinterpret_cast<const uint4*>(row + k);
        if (!raw_vec && live && g < steps) u = load_any(row, k, p.K);
        return u;
      };
#pragma unroll
      for (int j = 0; j < kQuad; ++j) word[j] = fetch(j);
      for (int g0 = 0, w = 0; g0 < steps && scales_free(w); g0 += kQuad, ++w) {
        const uint32_t scales = base + S::kScales + w % SQ * S::kScaleStage + 512;
#pragma unroll
        for (int j = 0; j < kQuad; ++j) {
          if (g0 + j >= steps || !stage_free(g0 + j)) break;
          const uint32_t to = base + (g0 + j) % ST * S::kStage + S::kA;
          const uint4 u = word[j];
          // The largest |value|, two bf16 at a time.
          uint32_t top = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                                  __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(~0u, top, o));
          const uint32_t e = scale_exponent(max(top << 16, top & 0xffff0000u));
          const float2 by = make_float2(inverse_scale(e), inverse_scale(e));
          const float2 v0 = mul2(bf16x2_to_float2(u.x), by), v1 = mul2(bf16x2_to_float2(u.y), by);
          const float2 v2 = mul2(bf16x2_to_float2(u.z), by), v3 = mul2(bf16x2_to_float2(u.w), by);
          asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(tile_at(to, r, piece >> 1) + (piece & 1) * 8),
                       "r"(pack_e4m3x2(v0.x, v0.y) | pack_e4m3x2(v1.x, v1.y) << 16),
                       "r"(pack_e4m3x2(v2.x, v2.y) | pack_e4m3x2(v3.x, v3.y) << 16)
                       : "memory");
          if (piece == 0)  // row r's word is the first of line r
            asm volatile("st.shared.u8 [%0], %1;" ::"r"(scales + r * 16 + j), "r"(e) : "memory");
          word[j] = fetch(g0 + j + kQuad);
        }
        if (!ok) break;
        fence_proxy_async_smem();
        warp_arrive(&bar.scale_full[w % SQ], lane);
      }
    }
  }
  __syncwarp();
  if (SPLIT && !kMeet) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // and so have the others
  if (warp < kEpilogueWarps && ok) ok = warp_wait(&bar.done, 0, abort);
  if (kMeet) cluster_sync_all();
  const int share = (NT + split - 1) / split;  // of the tile's tokens
  if (warp < kEpilogueWarps) {
    tc_fence_after();
    if (ok) {  // a lane is a channel, a column a token
      constexpr int C = 16;
      [[maybe_unused]] int owner = 0, t = 0;
#pragma unroll 1
      for (int c = 0; c < NT; c += C) {
        float v[C];
        tmem_ld16_nowait(tmem + ((uint32_t)(32 * warp) << 16) + c, v);
        tmem_ready(v);
#pragma unroll
        for (int j = 0; j < C; ++j) {
          if constexpr (SPLIT) {
            const uint32_t to = base + S::kParts + ((rank * share + t) * MT + 32 * warp + lane) * 4;
            st_cluster_f32(mapa_shared(to, owner), v[j]);
            if (++t == share) t = 0, ++owner;
          } else {
            const uint32_t to = base + S::kParts + ((c + j) * MT + 32 * warp + lane) * 4;
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(to), "f"(v[j]) : "memory");
          }
        }
      }
    }
  }
  if (!ok && lane == 0) {
    *abort = 1;
    atomicExch(p.status, kStatusTimeout);
  }
  // Given up: loads that were started arrive before the block ends.
  if (!ok && warp == kWarpLoad)
    for (int phase = 0; phase < 2; ++phase)
      for (int s = 0; s < ST; ++s) mbar_wait_bounded(&bar.full[s], phase, kWaitLimitCycles / 64);
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) tmem_dealloc(tmem, S::kTmemCols);
  if (SPLIT) cluster_sync_all();
  if (*abort) return;
  // This block's share, four channels a thread.
  const int first = m0 + rank * share, rows = min(min(share, NT - rank * share), p.M - first);
  Out* out = static_cast<Out*>(p.out) + (long long)first * p.N + n0;
  for (int id = threadIdx.x; id < rows * (MT / 4); id += kThreads<RAW>) {
    const int r = id / (MT / 4), c = id % (MT / 4) * 4, n = p.N - n0 - c;
    if (n <= 0) continue;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < split; ++s) {
      const uint4 u = ld_shared_v4(base + S::kParts + ((s * share + r) * MT + c) * 4);
      v.x += __uint_as_float(u.x), v.y += __uint_as_float(u.y);
      v.z += __uint_as_float(u.z), v.w += __uint_as_float(u.w);
    }
    Out* to = out + (long long)r * p.N + c;
    if constexpr (sizeof(Out) == 4) {
      if (vec) {
        *reinterpret_cast<float4*>(to) = v;
      } else {
        to[0] = v.x;
        if (n > 1) to[1] = v.y;
        if (n > 2) to[2] = v.z;
        if (n > 3) to[3] = v.w;
      }
    } else {
      if (vec) {
        *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      } else {
        to[0] = f_to_bf16(v.x);
        if (n > 1) to[1] = f_to_bf16(v.y);
        if (n > 2) to[2] = f_to_bf16(v.z);
        if (n > 3) to[3] = f_to_bf16(v.w);
      }
    }
  }
}

template <int NT, bool RAW, bool SPLIT, typename Out>
cudaError_t launch(const LinearProblem& p, int split, cudaStream_t stream) {
  using S = Smem<NT, SPLIT>;
  auto* kernel = linear_kernel<NT, RAW, SPLIT, Out>;
  // At every launch: the attribute belongs to the current device.
  const cudaError_t attr = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (attr != cudaSuccess) return attr;
  const EncodeTiledFn enc = tensor_map_encoder();
  CUtensorMap mw{}, mx{};
  if (!enc || !byte_map(enc, &mw, p.w, p.K, p.N, p.w_row, MT) ||
      (!RAW && !byte_map(enc, &mx, p.x, p.K, p.M, p.x_row, NT)))
    return cudaErrorNotSupported;
  const long long tokens = (p.M + NT - 1) / NT, tiles = tokens * ((p.N + MT - 1) / MT);
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)(tiles * split));
  c.blockDim = dim3(kThreads<RAW>);
  c.dynamicSmemBytes = S::kBytes;
  c.stream = stream;
  cudaLaunchAttribute a[2] = {};
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = (unsigned)split, a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
  a[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[1].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = a;
  c.numAttrs = p.follows ? 2 : 1;
  const bool raw_vec = RAW && aligned_to(p.raw, 16) && p.x_row % 8 == 0 && p.K % 8 == 0;
  const bool vec = p.N % 4 == 0 && aligned_to(p.out, 4 * sizeof(Out));
  return cudaLaunchKernelEx(&c, kernel, mw, mx, p, (int)tokens, split, raw_vec, vec);
}

template <int NT, bool RAW, typename Out>
cudaError_t run(const LinearProblem& p, cudaStream_t stream) {
  // As many blocks per tile as the SMs allow, each with a word of scales, four steps, at the least (64 and 128
  // tokens, 2048 x 1024: 5.8 and 7.7 us; with two steps each 7.1 and 9.5, the parts' sum costs more than it
  // saves; with the whole of K in a block 6.9 and 8.5, and 16.4 and 18.1 us instead of 7.5 and 8.7 for K = 8192).
  // A cluster's blocks lie within one of the GPU's graphics processing clusters, whose SMs do not divide evenly: no
  // more than so many clusters run at once, and a tile too many costs the whole time again (50 tiles in threes:
  // 30 us, in twos 23).
  static constexpr int kBlocks[] = {8, 6, 4, 3, 2}, kClusters[] = {15, 22, 36, 46, 76};
  const long long tiles = (long long)((p.M + NT - 1) / NT) * ((p.N + MT - 1) / MT);
  const int words = (scale_blocks(p.K) + kQuad - 1) / kQuad;
  int split = 1;
  for (int i = 0; i < 5 && split == 1; ++i)
    if (tiles <= kClusters[i] && kBlocks[i] <= words) split = kBlocks[i];
  return split > 1 ? launch<NT, RAW, true, Out>(p, split, stream) : launch<NT, RAW, false, Out>(p, 1, stream);
}

template <typename Out>
cudaError_t dispatch(const LinearProblem& p, cudaStream_t stream) {
  if (p.raw) return run<16, true, Out>(p, stream);
  if (p.M <= 16) return run<16, false, Out>(p, stream);
  if (p.M <= 32) return run<32, false, Out>(p, stream);
  if (p.M <= 64) return run<64, false, Out>(p, stream);
  return run<128, false, Out>(p, stream);
}

}  // namespace

cudaError_t launch_linear_fp8(const LinearProblem& p, cudaStream_t stream) {
  // More tiles of 128 x 128 than SMs would take another turn, where the larger tiles of pairs take one (2560 x 2048 x
  // 1024: 14.2 us here, 11.6 there; 2560 x 8192 x 1024: 34.9 and 24.7; one turn, 2048 x 2048 x 1024, is 8 and 11).
  const long long tiles = ((p.M + 127LL) / 128) * ((p.N + 127LL) / 128);
  if (p.M > 128 && tiles > 152) return launch_linear_pair(p, stream);
  return p.out_f32 ? dispatch<float>(p, stream) : dispatch<uint16_t>(p, stream);
}

}  // namespace m2rnn
