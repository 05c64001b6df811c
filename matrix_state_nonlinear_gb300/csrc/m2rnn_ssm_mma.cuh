// m2rnn_ssm_mma.cuh — shared by the chunked scan kernels: bf16 tiles in shared memory, their
// asynchronous loads, fragment loads and the split of a float32 value into two bf16 values.
#pragma once

#include "m2rnn_ssm.h"
#include "ptx_util.cuh"

namespace m2rnn {

// A tile of rows of kCols bf16 values (16, 32, 64 or 128), 16-byte chunks permuted within the
// rows so that eight rows' same chunk (an ldmatrix tile) falls on different banks.
template <int COLS>
struct Tile {
  static constexpr int kChunks = COLS / 8;
  static constexpr int kRowBytes = COLS * 2;
  __device__ __forceinline__ static uint32_t at(uint32_t base, int row, int chunk) {
    const int x = kChunks >= 8 ? row & 7 : kChunks == 4 ? (row >> 1) & 3 : (row >> 2) & 1;
    return base + row * kRowBytes + ((chunk ^ x) << 4);
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void st_shared_u16(uint32_t a, uint16_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(v) : "memory");
}
__device__ __forceinline__ void st_shared_u32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
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

// Starts the load of `rows` rows (of ROWS; the rest become zeros) of `width` values each, row r
// at src + r * stride, into a tile.  With `vec` (width % 8 == 0, 16-byte aligned rows) it is
// asynchronous; otherwise value by value, complete at the next block barrier.
template <int COLS, int ROWS, int THREADS>
__device__ __forceinline__ void load_tile(uint32_t tile, const uint16_t* src, long long stride, int rows,
                                          int width, bool vec, int tid) {
  constexpr int kChunks = Tile<COLS>::kChunks;
  if (vec) {
#pragma unroll
    for (int i = 0; i < (ROWS * kChunks + THREADS - 1) / THREADS; ++i) {
      const int id = tid + i * THREADS;
      if (ROWS * kChunks % THREADS != 0 && id >= ROWS * kChunks) break;
      const int row = id / kChunks, chunk = id % kChunks;
      const bool live = row < rows && chunk * 8 < width;
      cp_async16(Tile<COLS>::at(tile, row, chunk), live ? src + row * stride + chunk * 8 : src, live);
    }
  } else {
    for (int id = tid; id < ROWS * COLS; id += THREADS) {
      const int row = id / COLS, col = id % COLS;
      const uint16_t u = row < rows && col < width ? src[row * stride + col] : (uint16_t)0;
      st_shared_u16(Tile<COLS>::at(tile, row, col >> 3) + (col & 7) * 2, u);
    }
  }
}

// A operand (16 x 16): rows row0.., columns 8 chunk0.. of a tile.
template <int COLS>
__device__ __forceinline__ void frag_a(uint32_t (&r)[4], uint32_t tile, int row0, int chunk0, int lane) {
  ldsm_x4(r, Tile<COLS>::at(tile, row0 + (lane & 15), chunk0 + (lane >> 4)));
}
// A operand (16 x 16) of the transposed tile: A's rows are columns 8 chunk0.., its columns rows row0..
template <int COLS>
__device__ __forceinline__ void frag_at(uint32_t (&r)[4], uint32_t tile, int row0, int chunk0, int lane) {
  ldsm_x4_trans(r, Tile<COLS>::at(tile, row0 + (lane & 7) + ((lane >> 4) << 3), chunk0 + ((lane >> 3) & 1)));
}
// Two B operands (16 x 8 each) of X^T: B's columns are the tile's rows row0..+15 (n), its rows the
// tile's columns 8 chunk0..+15 (k).  r[0], r[1]: the first 8 columns; r[2], r[3]: the next 8.
template <int COLS>
__device__ __forceinline__ void frag_bn(uint32_t (&r)[4], uint32_t tile, int row0, int chunk0, int lane) {
  ldsm_x4(r, Tile<COLS>::at(tile, row0 + (lane & 7) + ((lane >> 4) << 3), chunk0 + ((lane >> 3) & 1)));
}
// Two B operands (16 x 8 each) of X: B's rows are the tile's rows row0..+15 (k), its columns the
// tile's columns 8 chunk0..+15 (n).
template <int COLS>
__device__ __forceinline__ void frag_bk(uint32_t (&r)[4], uint32_t tile, int row0, int chunk0, int lane) {
  ldsm_x4_trans(r, Tile<COLS>::at(tile, row0 + (lane & 15), chunk0 + (lane >> 4)));
}

// (x, y) as bf16 pairs hi + lo: hi is the rounding to bf16, lo that of the remainder, so that
// hi + lo is within 2^-17 of each value (2^-18 of its binade) and two bf16 products give nearly
// a float32 one.
__device__ __forceinline__ void split_bf16x2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x, y);
  lo = pack_bf16x2(x - bf16_lo(hi), y - bf16_hi(hi));
}

// The gates of a chunk's 64 tokens, by one warp (lane l has tokens l and l + 32), from their d
// and log2 f: sums over the chunk of log2 f, up to and including each token (cum) and after each
// token (rest; summed from the end, so that it stays exact where it matters, near zero).
struct ChunkSums {
  float cum0, cum1, rest0, rest1, total;
};
__device__ __forceinline__ ChunkSums chunk_sums(float l0, float l1, int lane) {
  float a = l0, b = l1, x = l0, y = l1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float pa = __shfl_up_sync(~0u, a, o), pb = __shfl_up_sync(~0u, b, o);
    const float px = __shfl_down_sync(~0u, x, o), py = __shfl_down_sync(~0u, y, o);
    if (lane >= o) a += pa, b += pb;
    if (lane + o < 32) x += px, y += py;
  }
  // x, y: suffix sums of each half, their own token included; exclusive by one shift.
  const float half0 = __shfl_sync(~0u, a, 31), half1 = __shfl_sync(~0u, y, 0);
  float ex = __shfl_down_sync(~0u, x, 1), ey = __shfl_down_sync(~0u, y, 1);
  if (lane == 31) ex = ey = 0.f;
  ChunkSums s;
  s.cum0 = a;
  s.cum1 = half0 + b;
  s.rest0 = ex + half1;
  s.rest1 = ey;
  s.total = half0 + half1;
  return s;
}

constexpr float kLog2e = 1.4426950408889634f;

}  // namespace m2rnn
