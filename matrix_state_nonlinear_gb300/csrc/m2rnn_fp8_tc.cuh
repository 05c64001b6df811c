// m2rnn_fp8_tc.cuh — 8-bit operands on the 5th-generation tensor cores, shared by the kernels of the
// projection: tensor maps, block-scaled products, scales in tensor memory.
//
// A stage holds 128 bytes of K, one scale block, of each row of both operands, 128-byte swizzled.  A
// product takes its scales from tensor memory, one byte of a 32-bit word per row, which its instruction
// names: a word holds the scales of four blocks one after the other, as they lie in memory, and scales are brought
// four words at a time, once in 16 stages (brought once a stage, each byte four times, they took longer than
// the products: 1040 us for 16384 x 4096 x 8192).  Words of rows 32 c .. 32 c + 31 of 128 are in column c, the same in
// each of the four quarters of the lanes.  They get there by a copy of 512 bytes of shared memory, line r
// holding the words of rows r, r + 32, r + 64, r + 96.
#pragma once

#include "m2rnn_internal.h"
#include "m2rnn_layer.h"
#include "m2rnn_ssm_tc.cuh"

namespace m2rnn {

constexpr int kBlockK = 128;  // bytes of K per stage

// Launches that overlap the one before: what the launch before has written may be read after this.
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}

// Instruction descriptor of kind::mxf8f6f4: e4m3 A and B (0), both K-major, scales of type e8m0 (bit 23),
// byte `which` of each scale word (bits 4 and 5 for B's, 29 and 30 for A's).
__host__ __device__ constexpr uint32_t idesc_fp8(int M, int N, uint32_t which) {
  return (which << 4) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24) | (which << 29);
}
// D (+)= (A sa)(B sb)^T over the 128 values of K of a stage, in four steps of 32, issued where `pred` holds: a
// whole warp runs the issuing loop, so that addresses and descriptors stay in uniform registers, and one
// lane issues.  (From a branch that one lane takes, the four products took 280 cycles to issue and a commit 118,
// of the 512 that the products themselves take.)  PAIR: across the two blocks of a pair.
template <bool PAIR>
__device__ __forceinline__ void umma4_fp8_if(bool pred, uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t sa, uint32_t sb, uint32_t accumulate_first) {
#define M2RNN_FP8_STEP(group, p)                                                                                   \
  "@q tcgen05.mma.cta_group::" group ".kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a, b, %3, [%4], [%5], " p ";\n\t"
#define M2RNN_FP8_STEPS(group)                                                                                     \
  "{\n\t.reg .pred p, q, t;\n\t.reg .b64 a, b;\n\t"                                                               \
  "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\tsetp.ne.b32 t, %8, 0;\n\tmov.b64 a, %1;\n\tmov.b64 b, %2;\n\t" \
  M2RNN_FP8_STEP(group, "p") "add.s64 a, a, 2;\n\tadd.s64 b, b, 2;\n\t" M2RNN_FP8_STEP(group, "t")               \
  "add.s64 a, a, 2;\n\tadd.s64 b, b, 2;\n\t" M2RNN_FP8_STEP(group, "t")                                          \
  "add.s64 a, a, 2;\n\tadd.s64 b, b, 2;\n\t" M2RNN_FP8_STEP(group, "t") "}"
  if constexpr (PAIR)
    asm volatile(M2RNN_FP8_STEPS("2")::"r"(d), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa), "r"(sb),
                 "r"(accumulate_first), "r"((int)pred), "r"(1)
                 : "memory");
  else
    asm volatile(M2RNN_FP8_STEPS("1")::"r"(d), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa), "r"(sb),
                 "r"(accumulate_first), "r"((int)pred), "r"(1)
                 : "memory");
#undef M2RNN_FP8_STEPS
#undef M2RNN_FP8_STEP
}
// Scales of 128 rows into 4 columns of tensor memory.  PAIR: the same copy in both blocks, each from its own
// shared memory.
template <bool PAIR>
__device__ __forceinline__ void copy_scales_if(bool pred, uint32_t tmem, uint32_t smem) {
  const uint64_t desc = umma_desc(smem, 0, 128, 0);
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(
            tmem),
        "l"(desc), "r"((int)pred)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(
            tmem),
        "l"(desc), "r"((int)pred)
        : "memory");
}
// A converged warp waits for a phase; the usual case, a phase that is over, costs one poll and no vote.
__device__ __forceinline__ bool issue_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  return warp_wait_long(smem_u32(bar), parity, abort);
}

constexpr int kQuad = 4;            // scale blocks, and stages, to a word
constexpr int kGroup = 4 * kQuad;  // and to a group of words

// Groups of scale words of ROWS rows per lane: the 16 blocks from i on, loaded one group ahead of their use,
// all loads before anything that waits for them.  Blocks behind a row's last get any scale: nothing uses them.
// A row of `blocks` scales starts anywhere, so a word of it is made of two whole words of memory; only words
// that hold a byte of the row are read, and of the rows whose words hold bytes outside the tensor (at most three
// at either end), where memory may end, bytes: those in one call a row after all other loads, as a call waits for
// its result (3840 x 3840 x 1280: 22.8 us with a call for each of the first and last row's words, 18.6 so).
template <int ROWS>
struct ScaleWords {
  const uint8_t* row[ROWS];
  bool live[ROWS], edge[ROWS];
  bool words;  // rows and their starts are whole words
  int blocks;  // of a row
  uint32_t next[ROWS][4], over[ROWS];
  // The tensor's row m of `rows`.
  __device__ __forceinline__ void aim(int r, const uint8_t* scales, long long m, long long rows) {
    live[r] = m < rows, edge[r] = live[r] && words_leave(scales, rows, blocks, m);
    row[r] = scales + m * blocks;
  }
  __device__ __forceinline__ void fetch(int i) {
    if (words) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          next[r][q] = 0x7f7f7f7fu;  // 1
          if (live[r] && i + 4 * q < blocks) next[r][q] = *reinterpret_cast<const uint32_t*>(row[r] + i + 4 * q);
        }
      return;
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int first = word_start(row[r], i);
#pragma unroll
      for (int q = 0; q < 5; ++q) {
        uint32_t w = 0x7f7f7f7fu;
        if (live[r] && !edge[r] && first + 4 * q < blocks) w = *reinterpret_cast<const uint32_t*>(row[r] + first + 4 * q);
        if (q < 4)
          next[r][q] = w;
        else
          over[r] = w;
      }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
      if (edge[r]) {
        const EdgeWords e = edge_words(row[r], word_start(row[r], i), blocks);
        next[r][0] = e.w[0], next[r][1] = e.w[1], next[r][2] = e.w[2], next[r][3] = e.w[3], over[r] = e.w[4];
      }
  }
  struct EdgeWords {
    uint32_t w[5];
  };
  // Five words from byte `first` of a row of `blocks` bytes on, zeros outside it.
  static __device__ __noinline__ EdgeWords edge_words(const uint8_t* row, int first, int blocks) {
    EdgeWords e;
#pragma unroll
    for (int q = 0; q < 5; ++q) {
      e.w[q] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = first + 4 * q + j;
        if (at >= 0 && at < blocks) e.w[q] |= (uint32_t)row[at] << (8 * j);
      }
    }
    return e;
  }
  // Word q of the group that was fetched from block i on.
  __device__ __forceinline__ uint32_t word(int r, int q, int i) const {
    if (words) return next[r][q];
    const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(row[r] + i) & 3u;
    return __funnelshift_r(next[r][q], q < 3 ? next[r][q < 3 ? q + 1 : 0] : over[r], 8 * off);
  }
};

// Tensor map of rows of K bytes in boxes of `rows` rows of 128 bytes, 128-byte swizzled; what lies outside
// is read as zero.
inline bool byte_map(EncodeTiledFn enc, CUtensorMap* map, const uint8_t* base, long long K, long long rows, long long row,
                     int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)row};
  const cuuint32_t box[2] = {(cuuint32_t)kBlockK, (cuuint32_t)box_rows}, estr[2] = {1u, 1u};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace m2rnn
