// m2rnn_ssm_tc.cuh — shared by the scan's kernels on the 5th-generation tensor cores.
//
// Operand tiles are bf16 in rows of 64 values (128 bytes), 128-byte swizzled (Tile<64>), a wider
// operand as panels of 64 columns.  An operand whose rows are the product's M (or N) is read
// K-major; one whose rows are the product's summed index is read MN-major.
#pragma once

#include "m2rnn_internal.h"
#include "m2rnn_ssm_mma.cuh"

namespace m2rnn {

// Byte offset of panel `i` of a tile of `rows` rows.
__device__ __forceinline__ constexpr int panel(int i, int rows) { return i * rows * 128; }

// D (+)= A B, A and B in shared memory, `steps` of 16 along the summed index; a and b are the
// descriptors of the first step, a_step and b_step their advance per step in 16-byte units, with
// an extra a_panel, b_panel after every fourth step (K-major panels; 0: none).
template <int STEPS, int A_STEP, int B_STEP, int A_PANEL = 0, int B_PANEL = 0>
__device__ __forceinline__ void umma_loop(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
#pragma unroll
  for (int i = 0; i < STEPS; ++i)
    umma_bf16(d, a + i * A_STEP + (i >> 2) * A_PANEL, b + i * B_STEP + (i >> 2) * B_PANEL, idesc,
              i > 0 || accumulate ? 1u : 0u);
}
// The same with A in tensor memory (16 bf16 values of a row in 8 columns).
__device__ __forceinline__ void umma_bf16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Descriptors of a swizzled tile at a 1024-byte aligned shared address: K-major, and MN-major with
// panels `rows` rows apart.
__device__ __forceinline__ uint64_t desc_k(uint32_t tile) { return umma_desc(tile, 16, 1024, 2); }
__device__ __forceinline__ uint64_t desc_mn(uint32_t tile, int rows) { return umma_desc(tile, rows * 128, 1024, 2); }

// Thread i of a warp reads (writes) 32 or 16 consecutive columns of tensor-memory lane i of the
// warp's quarter.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void st_shared_v4(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// A barrier of the whole block at which every thread learns whether any thread gave up.
__device__ __forceinline__ bool sync_or(bool bad) { return __syncthreads_or(bad); }

constexpr int kTokens = kSsmChunk;  // 128: a chunk is one row of every product per token

// What the products of a chunk need of its gates, per token.  Blocks are of 32 tokens.
struct alignas(16) ChunkGates {
  float cum[kTokens];   // log2 of the decay from the chunk's start, the token's own included
  float diag[kTokens];  // cum - log2 d: d exp(c_t - c_s) is 2^(cum_t - diag_s)
  float wd[kTokens];    // d times the decay from the token to the end of its block
  float wk[kTokens];    // d times the decay from the token to the chunk's end
  float total;          // log2 of the whole chunk's decay
};

// One warp fills a chunk's gates; lane l has tokens 4 l .. 4 l + 3, a their logits (-infinity past
// the sequence).  Sums over later tokens run from the end, so that they are exact near zero.
__device__ __forceinline__ void put_chunk_gates(ChunkGates& o, const float (&a)[4], float alpha, float beta, int lane) {
  float d[4], c[4], r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 g = ssm_gate(a[i], alpha, beta);
    d[i] = g.x, c[i] = r[i] = g.y * kLog2e;
  }
  c[1] += c[0], c[2] += c[1], c[3] += c[2];
  r[2] += r[3], r[1] += r[2], r[0] += r[1];
  float before = c[3], after = r[0];
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const float x = __shfl_up_sync(~0u, before, s), y = __shfl_down_sync(~0u, after, s);
    if (lane >= s) before += x;
    if (lane + s < 32) after += y;
  }
  const float total = __shfl_sync(~0u, before, 31);
  float pre = __shfl_up_sync(~0u, before, 1), post = __shfl_down_sync(~0u, after, 1);
  if (lane == 0) pre = 0.f;
  if (lane == 31) post = 0.f;
  const float end = __shfl_sync(~0u, pre + c[3], lane | 7);
  float4 cum, diag, wd, wk;
  float* pc = &cum.x;
  float* pd = &diag.x;
  float* pw = &wd.x;
  float* pk = &wk.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = pre + c[i];
    pc[i] = x;
    pd[i] = x - log2f(d[i]);
    pw[i] = d[i] * exp2_approx(end - x);
    pk[i] = d[i] * exp2_approx((i < 3 ? r[i + 1] : 0.f) + post);
  }
  reinterpret_cast<float4*>(o.cum)[lane] = cum;
  reinterpret_cast<float4*>(o.diag)[lane] = diag;
  reinterpret_cast<float4*>(o.wd)[lane] = wd;
  reinterpret_cast<float4*>(o.wk)[lane] = wk;
  if (lane == 0) o.total = total;
}

// Eight bf16 values as four float2.
__device__ __forceinline__ void unpack8(const uint4& u, float2 (&f)[4]) {
  f[0] = bf16x2_to_float2(u.x), f[1] = bf16x2_to_float2(u.y);
  f[2] = bf16x2_to_float2(u.z), f[3] = bf16x2_to_float2(u.w);
}

}  // namespace m2rnn
