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

// Loads tiles of ROWS rows of `width` values (the rest become zeros), row r at src + r * stride.
// With `vec` (width % 8 == 0, 16-byte aligned rows) the load is asynchronous; otherwise value by
// value, complete at the next block barrier.
template <int COLS, int ROWS, int THREADS>
struct TileLoader {
  static constexpr int kChunks = Tile<COLS>::kChunks;
  static constexpr int kStep = THREADS / kChunks;  // rows between a thread's pieces
  static constexpr int kPieces = (ROWS + kStep - 1) / kStep;
  static_assert(THREADS % kChunks == 0 && (kStep % 8 == 0 || kPieces == 1), "the same place in every row");
  const uint16_t *base, *src;  // row 0 of the sequence, and this thread's first piece
  long long stride;
  int row, width, col;
  uint32_t place;
  __device__ __forceinline__ void init(const uint16_t* base_, long long stride_, int width_, int tid) {
    base = base_, stride = stride_, width = width_;
    const int chunk = tid % kChunks;
    row = tid / kChunks, col = chunk * 8;
    place = Tile<COLS>::at(0, row, chunk);
    src = base + row * stride + col;
  }
  // Rows [t0, t0 + rows) of the sequence.
  __device__ __forceinline__ void load(uint32_t tile, long long t0, int rows, bool vec, int tid) const {
    if (vec) {
      const uint16_t* s = src + t0 * stride;
      const int most = col < width ? rows : 0;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        if (ROWS % kStep != 0 && row + i * kStep >= ROWS) break;
        const bool live = row + i * kStep < most;
        cp_async16(tile + place + i * kStep * Tile<COLS>::kRowBytes, live ? s : base, live);
        s += kStep * stride;
      }
    } else {
      const uint16_t* s = base + t0 * stride;
      for (int id = tid; id < ROWS * COLS; id += THREADS) {
        const int r = id / COLS, c = id % COLS;
        const uint16_t u = r < rows && c < width ? s[r * stride + c] : (uint16_t)0;
        st_shared_u16(Tile<COLS>::at(tile, r, c >> 3) + (c & 7) * 2, u);
      }
    }
  }
};

// A lane's part of the address of an ldmatrix of four 8 x 8 tiles, two down and two across a
// tile: `down` orders them down first, else across first.  A fragment at row row0 (a multiple
// of 8) and chunk chunk0 (even) is at tile + row0 * kRowBytes + (part ^ chunk0 * 16).
template <int COLS>
__device__ __forceinline__ uint32_t lane_part(int lane, bool down) {
  return down ? Tile<COLS>::at(0, lane & 15, lane >> 4)
              : Tile<COLS>::at(0, (lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
}
template <int COLS>
__device__ __forceinline__ uint32_t frag_at(uint32_t tile, uint32_t part, int row0, int chunk0) {
  return tile + row0 * Tile<COLS>::kRowBytes + (part ^ (chunk0 << 4));
}
// The fragments of m16n8k16 at such an address:
//   A (16 x 16), rows by columns of the tile:                      ldsm_x4,       part down
//   A of the transposed tile (A's rows are the tile's columns):    ldsm_x4_trans, part across
//   two B (16 x 8) of the tile, k its rows, n its columns:         ldsm_x4_trans, part down
//   two B of the transposed tile, k its columns, n its rows:       ldsm_x4,       part across
// Of two B fragments r[0], r[1] are the first 8 columns (n), r[2], r[3] the next 8.

// (x, y) as bf16 pairs hi + lo: hi is the rounding to bf16, lo that of the remainder, so that
// hi + lo is within 2^-17 of each value (2^-18 of its binade) and two bf16 products give nearly
// a float32 one.
__device__ __forceinline__ void split_bf16x2(float2 x, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x.x, x.y);
  const float2 r = sub2(x, bf16x2_to_float2(hi));
  lo = pack_bf16x2(r.x, r.y);
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

// A state (or its gradient) of KP x VT float32 values over the accumulators of four warps: MT
// tiles of 16 rows by NT tiles of 8 columns each.  A warp of a state with fewer than four row
// tiles takes some of the columns.
template <int KP, int VT>
struct StateTiles {
  static constexpr int kRowTiles = KP / 16;
  static constexpr bool kSplit = kRowTiles < 4;
  static constexpr int MT = kSplit ? 1 : kRowTiles / 4;
  static constexpr int NT = kSplit ? VT / 8 * kRowTiles / 4 : VT / 8;
  __device__ static int row_tile(int warp) { return kSplit ? warp % kRowTiles : warp * MT; }
  __device__ static int col_tile(int warp) { return kSplit ? warp / kRowTiles * NT : 0; }
};

template <typename T>
__device__ __forceinline__ void scale_state(float (&H)[T::MT][T::NT][4], float f) {
  const float2 f2 = make_float2(f, f);
#pragma unroll
  for (int m = 0; m < T::MT; ++m)
#pragma unroll
    for (int j = 0; j < T::NT; ++j)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 h = mul2(make_float2(H[m][j][2 * r], H[m][j][2 * r + 1]), f2);
        H[m][j][2 * r] = h.x, H[m][j][2 * r + 1] = h.y;
      }
}

// H += sum over the 16 tokens t of block j of (w[t] x_t) y_t^T: x from its tile [token][KP], y as
// the B fragments of those tokens.  w x is split into two bf16 values.
template <int KP, typename T>
__device__ __forceinline__ void add_outer(float (&H)[T::MT][T::NT][4], uint32_t tile_x, uint32_t part_x,
                                          const float* w, const uint32_t (&yf)[4][4], int j, int m0, int nt0,
                                          int c2) {
  const float2 w0 = *reinterpret_cast<const float2*>(w + j * 16 + c2);
  const float2 w1 = *reinterpret_cast<const float2*>(w + j * 16 + 8 + c2);
#pragma unroll
  for (int m = 0; m < T::MT; ++m) {
    uint32_t xf[4], hi[4], lo[4];
    ldsm_x4_trans(xf, frag_at<KP>(tile_x, part_x, j * 16, (m0 + m) * 2));
#pragma unroll
    for (int r = 0; r < 4; ++r) split_bf16x2(mul2(bf16x2_to_float2(xf[r]), r < 2 ? w0 : w1), hi[r], lo[r]);
#pragma unroll
    for (int i = 0; i < T::NT; ++i) {
      uint32_t b0 = yf[i >> 1][(i & 1) * 2], b1 = yf[i >> 1][(i & 1) * 2 + 1];
      if constexpr (T::kSplit) {  // column tile nt0 + i, chosen without indexing registers
#pragma unroll
        for (int o = 0; o < 8; ++o)
          if (o == nt0 + i) b0 = yf[o >> 1][(o & 1) * 2], b1 = yf[o >> 1][(o & 1) * 2 + 1];
      }
      mma_bf16_16816(H[m][i], hi, b0, b1);
      mma_bf16_16816(H[m][i], lo, b0, b1);
    }
  }
}

}  // namespace m2rnn
