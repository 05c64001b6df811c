// m2rnn_linear.cu — product of 8-bit activations and weights with block scales.
//
//   out[m, n] = sum_k x[m, k] sx[m, k / 128] w[n, k] sw[n / 128, k / 128]
//
// The scales are powers of two, so the tensor cores apply them exactly (kind::mxf8f6f4) and the sum over
// all of K stays in one float32 accumulator in tensor memory.
#include "m2rnn_internal.h"
#include "m2rnn_layer.h"
#include "m2rnn_ssm_tc.cuh"

namespace m2rnn {
namespace {

constexpr int MT = 128;  // output channels of a tile: the product's rows (tensor-memory lanes)
constexpr int KB = 128;  // bytes of K per stage: one scale block
constexpr int kEpilogueWarps = 4, kWarpLoad = 4, kWarpMma = 5, kWarpScale = 6, kThreads = 224;

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}

// Instruction descriptor of kind::mxf8f6f4: e4m3 A and B (0), both K-major, scales of type e8m0 (bit 23),
// the first byte of each scale word.
__host__ __device__ constexpr uint32_t idesc_fp8(int M, int N) {
  return ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24);
}
// D (+)= (A sa)(B sb)^T over 32 values of K.
__device__ __forceinline__ void umma_fp8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
      : "memory");
}
// Scales of 128 rows into 4 columns of tensor memory: word c of 16-byte line r is that of row 32 c + r.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint32_t smem) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(umma_desc(smem, 0, 128, 0))
               : "memory");
}

template <int NT>
struct Smem {
  static constexpr int kStages = 5;
  static constexpr int kA = MT * KB, kB = NT * KB, kStage = kA + kB;
  static constexpr int kScales = kStages * kStage, kScaleStage = 1024;
  static constexpr int kBytes = kScales + kStages * kScaleStage + 1024;  // 1024: to align the first stage
};
template <int S>
struct Bars {
  uint64_t full[S], empty[S], done;
  uint32_t tmem;
  int abort;
};

template <int NT, typename Out>
__global__ void __launch_bounds__(kThreads)
    linear_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, LinearProblem p,
                  int token_tiles, bool vec) {
  using S = Smem<NT>;
  constexpr int ST = S::kStages;
  extern __shared__ unsigned char raw[];
  __shared__ Bars<ST> bar;
  unsigned char* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = (int)(blockIdx.x / token_tiles) * MT, m0 = (int)(blockIdx.x % token_tiles) * NT;
  const int blocks = scale_blocks(p.K);
  volatile int* abort = &bar.abort;
  constexpr int kTmemCols = 256, kColScale = NT;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) mbar_init(&bar.full[s], 2), mbar_init(&bar.empty[s], 1);
    mbar_init(&bar.done, 1);
    bar.abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc(&bar.tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;
  bool ok = true;

  if (warp == kWarpLoad) {
    for (int i = 0; i < blocks; ++i) {
      const int s = i % ST;
      if (i >= ST && !(ok = warp_wait(&bar.empty[s], (uint32_t)(i / ST - 1) & 1u, abort))) break;
      if (lane == 0) {
        unsigned char* to = smem + s * S::kStage;
        mbar_arrive_expect_tx(&bar.full[s], S::kStage);
        tma_load_2d(to, &map_w, &bar.full[s], i * KB, n0);
        tma_load_2d(to + S::kA, &map_x, &bar.full[s], i * KB, m0);
      }
      __syncwarp();
    }
  } else if (warp == kWarpScale) {
    const uint8_t* sw = p.w_scales + (size_t)(n0 / KB) * blocks;
    for (int i = 0; i < blocks; ++i) {
      const int s = i % ST;
      uint32_t u[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int m = m0 + 32 * c + lane;
        u[c] = (32 * c < NT && m < p.M ? p.x_scales[(size_t)m * blocks + i] : 127u) * 0x01010101u;
      }
      const uint32_t v = sw[i] * 0x01010101u;
      if (i >= ST && !(ok = warp_wait(&bar.empty[s], (uint32_t)(i / ST - 1) & 1u, abort))) break;
      const uint32_t to = base + S::kScales + s * S::kScaleStage;
      st_shared_v4(to + lane * 16, make_uint4(v, v, v, v));
      st_shared_v4(to + 512 + lane * 16, make_uint4(u[0], u[1], u[2], u[3]));
      fence_proxy_async_smem();
      warp_arrive(&bar.full[s], lane);
    }
  } else if (warp == kWarpMma) {
    constexpr uint32_t idesc = idesc_fp8(MT, NT);
    for (int i = 0; i < blocks; ++i) {
      const int s = i % ST;
      if (!(ok = warp_wait(&bar.full[s], (uint32_t)(i / ST) & 1u, abort))) break;
      tc_fence_after();
      if (lane == 0) {
        const uint32_t at = base + s * S::kStage, scales = base + S::kScales + s * S::kScaleStage;
        const uint32_t sa = tmem + kColScale + 8 * s, sb = sa + 4;
        copy_scales(sa, scales);
        copy_scales(sb, scales + 512);
        const uint64_t a = desc_k(at), b = desc_k(at + S::kA);
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_fp8(tmem, a + 2 * k, b + 2 * k, idesc, sa, sb, i > 0 || k > 0);
        umma_commit(&bar.empty[s]);
        if (i == blocks - 1) umma_commit(&bar.done);
      }
      __syncwarp();
    }
  } else {
    ok = warp_wait(&bar.done, 0, abort);
    tc_fence_after();
    // Lane = channel: a tile row by row (token) through the stages, which every product has left.
    Out* tile = reinterpret_cast<Out*>(smem);
    if (ok) {
#pragma unroll 1
      for (int c = 0; c < NT; c += 16) {
        float v[16];
        tmem_ld16_nowait(tmem + ((uint32_t)(32 * warp) << 16) + c, v);
        tmem_ready(v);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          Out* to = tile + (c + j) * MT + 32 * warp + lane;
          if constexpr (sizeof(Out) == 4)
            *to = v[j];
          else
            *to = f_to_bf16(v[j]);
        }
      }
    }
    named_bar_sync(1, 32 * kEpilogueWarps);
    if (ok) {
      const int rows = min(NT, p.M - m0), width = min(MT, p.N - n0);
      Out* out = static_cast<Out*>(p.out) + (size_t)m0 * p.N + n0;
      if (vec) {
        constexpr int V = 16 / sizeof(Out), L = MT / V;  // values per access, accesses per row
        for (int id = threadIdx.x; id < rows * L; id += 32 * kEpilogueWarps) {
          const int r = id / L, c = id % L * V;
          if (c < width)
            *reinterpret_cast<uint4*>(out + (size_t)r * p.N + c) = *reinterpret_cast<const uint4*>(tile + r * MT + c);
        }
      } else {
        for (int id = threadIdx.x; id < rows * MT; id += 32 * kEpilogueWarps) {
          const int r = id / MT, c = id % MT;
          if (c < width) out[(size_t)r * p.N + c] = tile[r * MT + c];
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
  if (warp == kWarpMma) tmem_dealloc(tmem, kTmemCols);
}

// Tensor map of rows of K bytes in boxes of `rows` rows of 128 bytes, 128-byte swizzled; what lies outside
// is read as zero.
bool byte_map(EncodeTiledFn enc, CUtensorMap* map, const uint8_t* base, long long K, long long rows, long long row,
              int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)row};
  const cuuint32_t box[2] = {(cuuint32_t)KB, (cuuint32_t)box_rows}, estr[2] = {1u, 1u};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, typename Out>
cudaError_t run(const LinearProblem& p, cudaStream_t stream) {
  using S = Smem<NT>;
  // At every launch: the attribute belongs to the current device.
  const cudaError_t attr =
      cudaFuncSetAttribute(linear_kernel<NT, Out>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (attr != cudaSuccess) return attr;
  const EncodeTiledFn enc = tensor_map_encoder();
  CUtensorMap mw{}, mx{};
  if (!enc || !byte_map(enc, &mw, p.w, p.K, p.N, p.w_row, MT) || !byte_map(enc, &mx, p.x, p.K, p.M, p.x_row, NT))
    return cudaErrorNotSupported;
  const long long tokens = (p.M + NT - 1) / NT, channels = (p.N + MT - 1) / MT;
  const bool vec = p.N % (16 / (int)sizeof(Out)) == 0 && aligned_to(p.out, 16);
  linear_kernel<NT, Out><<<(unsigned)(tokens * channels), kThreads, S::kBytes, stream>>>(mw, mx, p, (int)tokens, vec);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_fp8(const LinearProblem& p, cudaStream_t stream) {
  return p.out_f32 ? run<128, float>(p, stream) : run<128, uint16_t>(p, stream);
}

}  // namespace m2rnn
