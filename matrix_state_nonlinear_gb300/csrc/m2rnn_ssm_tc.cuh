// m2rnn_ssm_tc.cuh — shared by the scan's kernels on the 5th-generation tensor cores.
//
// Operand tiles are bf16 in rows of 64 values (128 bytes), 128-byte swizzled (tile_at), a wider
// operand as panels of 64 columns.  An operand whose rows are the product's M (or N) is read
// K-major; one whose rows are the product's summed index is read MN-major.
#pragma once

#include "m2rnn_internal.h"
#include "m2rnn_ssm.h"
#include "ptx_util.cuh"

namespace m2rnn {

constexpr float kLog2e = 1.4426950408889634f;

// Shared address of 16-byte chunk `chunk` of row `row` of a tile of rows of 64 bf16 values: chunks are
// permuted within a row as the 128-byte swizzle has them.
__device__ __forceinline__ uint32_t tile_at(uint32_t tile, int row, int chunk) {
  return tile + row * 128 + ((chunk ^ (row & 7)) << 4);
}
__device__ __forceinline__ void st_shared_u16(uint32_t a, uint16_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
// 2^x, at most 2 ulp off.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// (x, y) as bf16 pairs hi + lo: hi is the rounding to bf16, lo that of the remainder, so that
// hi + lo is within 2^-17 of each value (2^-18 of its binade) and two bf16 products give nearly
// a float32 one.
__device__ __forceinline__ void split_bf16x2(float2 x, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x.x, x.y);
  const float2 r = sub2(x, bf16x2_to_float2(hi));
  lo = pack_bf16x2(r.x, r.y);
}

// Byte offset of panel `i` of a tile of `rows` rows.
__device__ __forceinline__ constexpr int panel(int i, int rows) { return i * rows * 128; }

// D (+)= A B over STEPS (a multiple of four) steps of 16 along the summed index, issued where
// `pred` holds; a and b describe the first step, A_STEP and B_STEP are their advance per step and
// A_PANEL, B_PANEL the further advance after every fourth (16-byte units).
template <int STEPS, int A_STEP, int B_STEP, int A_PANEL = 0, int B_PANEL = 0>
__device__ __forceinline__ void umma_steps(bool pred, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           bool accumulate) {
#pragma unroll 1
  for (int i = 0; i < STEPS / 4; ++i)
    umma4_if<A_STEP, B_STEP>(pred, d, a + i * (4 * A_STEP + A_PANEL), b + i * (4 * B_STEP + B_PANEL), idesc,
                             i > 0 || accumulate ? 1u : 0u);
}
// Four steps with A in tensor memory (16 bf16 values of a row in 8 columns).
template <int B_STEP>
__device__ __forceinline__ void umma4_ta_if(bool pred, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate_first) {
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\tsetp.ne.b32 t, %7, 0;\n\t"
      "mov.b32 a, %1;\n\tmov.b64 b, %2;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p;\n\t"
      "add.s32 a, a, 8;\n\tadd.s64 b, b, %6;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.s32 a, a, 8;\n\tadd.s64 b, b, %6;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.s32 a, a, 8;\n\tadd.s64 b, b, %6;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate_first), "r"((int)pred), "n"(B_STEP), "r"(1)
      : "memory");
}

// Descriptors of a swizzled tile at a 1024-byte aligned shared address: K-major, and MN-major with
// panels `rows` rows apart.
__device__ __forceinline__ uint64_t desc_k(uint32_t tile) { return umma_desc(tile, 16, 1024, 2); }
__device__ __forceinline__ uint64_t desc_mn(uint32_t tile, int rows) { return umma_desc(tile, rows * 128, 1024, 2); }

// Waits for the warp's loads from tensor memory into v...  The empty statements tie every later use
// of the registers to the wait: without them the compiler may move arithmetic on them before it.
template <int N>
__device__ __forceinline__ void tie(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
template <typename... V>
__device__ __forceinline__ void tmem_ready(V&... v) {
  tmem_wait_ld();
  (tie(v), ...);
}
// Thread i of a warp loads 8 consecutive columns of tensor-memory lane i of the warp's quarter.
__device__ __forceinline__ void tmem_ld8_nowait(uint32_t taddr, float (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "r"(taddr));
}
// Thread i of a warp writes 8 consecutive columns of tensor-memory lane i of the warp's quarter.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void st_shared_v4(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// warp_wait in full: one copy for all the warps' programs, which compete for the instruction cache.
static __device__ __noinline__ bool warp_wait_long(uint32_t bar, uint32_t parity, volatile int* abort) {
  const uint32_t start = (uint32_t)clock();
  uint32_t done;
  do {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (!done && (*abort || (uint32_t)clock() - start > (uint32_t)kWaitLimitCycles)) break;
  } while (!done);
  return __all_sync(~0u, done != 0);
}
// A whole warp waits for the phase of `bar` with the given parity; false, for every lane, where the
// wait ran out or another warp has given up.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (__all_sync(~0u, mbar_try_wait(bar, parity))) return true;
  return warp_wait_long(smem_u32(bar), parity, abort);
}
// One arrival for the warp, after its lanes' earlier work.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Copies `bytes` (a multiple of 16) of consecutive memory into shared memory; completion as
// transaction bytes on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// Starts the fetch of a box into L2, where a later load will find it.
__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap* map, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}

// Tensor map of a bf16 operand [B][T][heads][width] with free token and batch strides, in boxes of
// 128 tokens by 64 columns of one head, 128-byte swizzled; what lies outside is read as zero.
inline bool token_map(EncodeTiledFn enc, CUtensorMap* map, const uint16_t* base, int width, int heads, int T, int B,
                      const Strides& s) {
  const cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)width * 2, (cuuint64_t)s.token * 2, (cuuint64_t)s.batch * 2};
  const cuuint32_t box[4] = {64u, 1u, (cuuint32_t)kSsmChunk, 1u};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return s.token > 0 && s.batch > 0 &&
         enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The same box by one warp, value by value, for operands that a tensor map cannot describe.
static __device__ __noinline__ void copy_tokens(uint32_t tile, const uint16_t* src, long long stride, int rows,
                                                int width, int lane) {
  for (int id = lane; id < kSsmChunk * 64; id += 32) {
    const int r = id >> 6, c = id & 63;
    st_shared_u16(tile_at(tile, r, c >> 3) + (c & 7) * 2,
                  r < rows && c < width ? src[r * stride + c] : (uint16_t)0);
  }
}

constexpr int kTokens = kSsmChunk;  // 128: a chunk is one row of every product per token

// Tensor map of kept states [pairs][planes][K][V] in boxes of kp rows of 64 columns of one plane.
inline bool state_map(EncodeTiledFn enc, CUtensorMap* map, const uint16_t* base, int K, int V, long long planes,
                      long long pairs, int kp) {
  const cuuint64_t dims[4] = {(cuuint64_t)V, (cuuint64_t)K, (cuuint64_t)planes, (cuuint64_t)pairs};
  const cuuint64_t strides[3] = {(cuuint64_t)V * 2, (cuuint64_t)K * V * 2, (cuuint64_t)K * V * 2 * planes};
  const cuuint32_t box[4] = {64u, (cuuint32_t)kp, 1u, 1u};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// A state's two planes [K][V] into two tiles of KP rows, by one warp, value by value.
template <int KP>
__device__ __forceinline__ void copy_state(uint32_t tile, const uint16_t* src, int K, int V, int width, int lane) {
  for (int id = lane; id < 2 * KP * 64; id += 32) {
    const int x = id / (KP * 64), r = id / 64 % KP, c = id % 64;
    st_shared_u16(tile_at(tile + x * KP * 128, r, c >> 3) + (c & 7) * 2,
                  r < K && c < width ? src[((size_t)x * K + r) * V + c] : (uint16_t)0);
  }
  fence_proxy_async_smem();
}
// One warp copies tokens of a swizzled tile to memory, value by value: row r to dst + r * stride.
__device__ __forceinline__ void copy_out(uint16_t* dst, uint32_t tile, long long stride, int rows, int width, int lane) {
  for (int id = lane; id < kSsmChunk * 64; id += 32) {
    const int r = id >> 6, c = id & 63;
    if (r < rows && c < width) {
      const uint32_t u = ld_shared_u32(tile_at(tile, r, c >> 3) + (c & 6) * 2);
      dst[r * stride + c] = (uint16_t)(c & 1 ? u >> 16 : u);
    }
  }
}

// What the products of a chunk need of its gates.  Blocks are of 32 tokens; B_t is log2 of the decay from
// the start of a token's block to the token, its own included.
//
// Between tokens s < t of two blocks the weight exp(c_t - c_s) d_s is 2^(B_t + span of the blocks between)
// wd_s, within a block it is 2^(B_t - B_s) d_s.  B is kept as hi + lo.  Where a block decays by 2^-256 or
// more in all, hi sums each token's log2 f rounded to a multiple of 2^-8, exactly (a block's sum is below
// 2^13, as log f is held at -105 and above), and lo the rests, which stay below 1/16: B_t - B_s taken part
// by part is then as exact as a sum over the tokens from s to t alone.  In one float it would lose 2^-24 of
// B itself, 3e-4 of a weight between the last tokens of a block whose others forget the state (and 1.7e-3
// summed from the chunk's start).  In any other block, nearly every one, hi is zero and lo is B, within
// 2^-16 of a weight, and the usual path needs lo alone.
struct alignas(16) ChunkGates {
  float hi[kTokens], lo[kTokens];
  float diag[kTokens];  // lo - log2 d: d exp(c_t - c_s) is 2^((hi_t - hi_s) + (lo_t - diag_s)) within a block
  float wd[kTokens];    // d times the decay from the token to the end of its block
  float wk[kTokens];    // d times the decay from the token to the chunk's end
  float span[5][4];     // [i][j], j <= i: log2 of the decay of blocks j .. i - 1
  __device__ __forceinline__ float total() const { return span[4][0]; }  // log2 of the whole chunk's decay
  // log2 of the decay from the chunk's start to a token, its own included.
  __device__ __forceinline__ float from_start(int t) const { return (hi[t] + lo[t]) + span[t >> 5][0]; }
  // Whether a block's tokens differ in hi (which, like B, only falls or only rises).
  __device__ __forceinline__ bool wide(int block) const { return hi[32 * block + 31] != 0.f; }
};

// One warp fills a chunk's gates; `logits` gives the logit of a token of the chunk (-infinity past
// the sequence).  Each token's own values first (in o's arrays), then lane l sums over tokens
// 4 l .. 4 l + 3 and the lanes before.  The loop is kept short on purpose: the block's warps run
// different code, and what does not fit the instruction cache stalls them all.
template <typename Logits>
__device__ __forceinline__ void put_chunk_gates(ChunkGates& o, Logits logits, float alpha, float beta, int lane) {
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const int t = 32 * i + lane;
    const float2 g = ssm_gate(logits(i), alpha, beta);
    const float c = g.y * kLog2e, h = (c + 49152.f) - 49152.f;  // 1.5 * 2^15: one ulp is 2^-8
    o.wd[t] = g.x;
    o.hi[t] = h;
    o.lo[t] = c - h;
    o.diag[t] = log2f(g.x);
  }
  __syncwarp();
  float4 h = reinterpret_cast<const float4*>(o.hi)[lane], l = reinterpret_cast<const float4*>(o.lo)[lane];
  h.y += h.x, h.z += h.y, h.w += h.z;
  l.y += l.x, l.z += l.y, l.w += l.z;
  float sh = h.w, sl = l.w;  // over the block's lanes up to this one
#pragma unroll
  for (int s = 1; s < 8; s <<= 1) {
    const float x = __shfl_up_sync(~0u, sh, s, 8), y = __shfl_up_sync(~0u, sl, s, 8);
    if ((lane & 7) >= s) sh += x, sl += y;
  }
  const float eh = __shfl_sync(~0u, sh, 7, 8), el = __shfl_sync(~0u, sl, 7, 8);  // over the block
  sh -= h.w, sl -= l.w;  // before the lane
  h = make_float4(sh + h.x, sh + h.y, sh + h.z, sh + h.w);
  l = make_float4(sl + l.x, sl + l.y, sl + l.z, sl + l.w);
  const float4 d = reinterpret_cast<const float4*>(o.wd)[lane], ld = reinterpret_cast<const float4*>(o.diag)[lane];
  const float4 wd = make_float4(d.x * exp2_approx((eh - h.x) + (el - l.x)), d.y * exp2_approx((eh - h.y) + (el - l.y)),
                                d.z * exp2_approx((eh - h.z) + (el - l.z)), d.w * exp2_approx((eh - h.w) + (el - l.w)));
  reinterpret_cast<float4*>(o.wd)[lane] = wd;
  if (fabsf(eh) < 256.f) {
    l = make_float4(l.x + h.x, l.y + h.y, l.z + h.z, l.w + h.w);
    h = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  reinterpret_cast<float4*>(o.hi)[lane] = h;
  reinterpret_cast<float4*>(o.lo)[lane] = l;
  reinterpret_cast<float4*>(o.diag)[lane] = make_float4(l.x - ld.x, l.y - ld.y, l.z - ld.z, l.w - ld.w);
  // Sums over whole blocks: of the later ones for wk, and span[i][j] by lane 4 i + j.
  const uint32_t later = 14u << (lane >> 3), part = ((1u << (lane >> 2)) - 1u) & (15u << (lane & 3));
  float tail = 0.f, span = 0.f;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const float x = __shfl_sync(~0u, eh + el, 8 * b);
    if (later >> b & 1) tail += x;
    if (part >> b & 1) span += x;
  }
  const float e = exp2_approx(tail);
  reinterpret_cast<float4*>(o.wk)[lane] = make_float4(e * wd.x, e * wd.y, e * wd.z, e * wd.w);
  if (lane < 20) o.span[0][lane] = span;
}

// Eight bf16 values as four float2.
__device__ __forceinline__ void unpack8(const uint4& u, float2 (&f)[4]) {
  f[0] = bf16x2_to_float2(u.x), f[1] = bf16x2_to_float2(u.y);
  f[2] = bf16x2_to_float2(u.z), f[3] = bf16x2_to_float2(u.w);
}

}  // namespace m2rnn
