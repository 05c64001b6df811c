// m2rnn_groupnorm.cu — gated group norm over the channels of one token, and its backward.
//
//   n = (y - mean) inv,  inv = 1 / sqrt(var + eps),  p = w n + b
//   out = p s(g)  (s = SiLU, with a gate)   or   out = s(p)  (without)
// Backward, with dp = dout s(g) or dout s'(p):
//   dg = dout p s'(g),  dw = sum dp n,  db = sum dp,  dn = dp w
//   dy = inv (dn - mean(dn) - n mean(dn n))
//
// Memory-bound: the forward moves 6 bytes an element, the backward 10 (bf16, with a gate).  A
// team of lanes takes one group of one row: each lane holds its share in registers, so y is read
// once, and mean and variance are two exact passes over registers (the variance of the centred
// values; no sum of squares is subtracted).  A team is 8, 16 or 32 lanes of a warp, or the whole
// block for groups of more than 32 lanes' registers.  Short groups' forward loads three rows per team
// before it computes the first; the backward keeps a team on the same channels for many rows,
// the next row loaded while one is computed, so that dw and db add up in registers and one row
// of partial sums per team goes to memory.  All arithmetic is on pairs: at one value an
// instruction both directions were bound by instruction issue (206 and 354 us).
// Measured, 131072 rows of 16 groups of 64, bf16 with a gate: forward 136 us (5.9 TB/s, 87 % of a copy),
// backward 228 us (5.9 TB/s) and 6 us for the sums.
#include "m2rnn_ssm.h"
#include "ptx_util.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 256;

// VEC values (8 or 1) as loaded, so that a load can be started ahead of its use, and as PAIRS
// float pairs (of which VEC = 1 uses one half, the other is zero).
template <int VEC>
constexpr int kPairs = VEC == 8 ? 4 : 1;
template <typename Y, int VEC>
struct Raw {
  uint4 u[VEC == 8 && sizeof(Y) == 4 ? 2 : 1];
  __device__ __forceinline__ void load(const Y* p) {
    if constexpr (VEC == 8) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(Y) / 2; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
    } else if constexpr (sizeof(Y) == 4) {
      u[0].x = __float_as_uint(*p);
    } else {
      u[0].x = *p;
    }
  }
  __device__ __forceinline__ void get(float2 (&f)[kPairs<VEC>]) const {
    if constexpr (VEC == 8 && sizeof(Y) == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[2 * i] = make_float2(__uint_as_float(u[i].x), __uint_as_float(u[i].y));
        f[2 * i + 1] = make_float2(__uint_as_float(u[i].z), __uint_as_float(u[i].w));
      }
    } else if constexpr (VEC == 8) {
      f[0] = bf16x2_to_float2(u[0].x), f[1] = bf16x2_to_float2(u[0].y);
      f[2] = bf16x2_to_float2(u[0].z), f[3] = bf16x2_to_float2(u[0].w);
    } else {
      f[0] = make_float2(sizeof(Y) == 4 ? __uint_as_float(u[0].x) : bf16_to_f((uint16_t)u[0].x), 0.f);
    }
  }
};

template <int VEC>
__device__ __forceinline__ void store_vals(uint16_t* p, const float2 (&f)[kPairs<VEC>]) {
  if constexpr (VEC == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y),
                                              pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y));
  else
    *p = f_to_bf16(f[0].x);
}
template <int VEC>
__device__ __forceinline__ void store_vals(float* p, const float2 (&f)[kPairs<VEC>]) {
  if constexpr (VEC == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
  } else {
    *p = f[0].x;
  }
}

__device__ __forceinline__ float2 pair(float x) { return make_float2(x, x); }

// Sums over the team, TEAM lanes of a warp or (TEAM 0) the whole block, two values at once.
// Every thread of the block calls it (lanes without a group pass zeros).
template <int TEAM>
__device__ __forceinline__ float2 team_sum(float2 s) {
#pragma unroll
  for (int o = (TEAM ? TEAM : 32) / 2; o > 0; o >>= 1)
    s = add2(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, s.y, o)));
  if constexpr (!TEAM) {
    __shared__ float2 part[kThreads / 32];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s = add2(s, part[w]);
    __syncthreads();
  }
  return s;
}
template <int TEAM>
__device__ __forceinline__ float team_sum(float s) {
  if constexpr (!TEAM) {
    return team_sum<0>(make_float2(s, 0.f)).x;
  } else {
#pragma unroll
    for (int o = TEAM / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  }
}

// This thread's share of a group: chunks lane, lane + width, ... of VEC values each.
template <int TEAM>
struct Lanes {
  static constexpr int kWidth = TEAM ? TEAM : kThreads;
  static __device__ __forceinline__ int lane() { return threadIdx.x & (kWidth - 1); }
  static __device__ __forceinline__ long long team() {
    return TEAM ? ((long long)blockIdx.x * kThreads + threadIdx.x) / kWidth : blockIdx.x;
  }
};

// Centres and scales a group's values (zeros outside it): z becomes n; returns inv.
template <int VEC, int TEAM, int R>
__device__ __forceinline__ float normalise(bool live, int chunks, float inv_e, float eps,
                                           float2 (&z)[R][kPairs<VEC>]) {
  constexpr int P = kPairs<VEC>;
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < P; ++i) s = add2(s, z[r][i]);
  const float2 mean = pair(team_sum<TEAM>(s.x + s.y) * inv_e);
  s = make_float2(0.f, 0.f);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (live && Lanes<TEAM>::lane() + r * Lanes<TEAM>::kWidth < chunks) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        z[r][i] = sub2(z[r][i], mean);
        if (VEC == 1) z[r][i].y = 0.f;
        s = fma2(z[r][i], z[r][i], s);
      }
    }
  }
  const float inv = rsqrtf(team_sum<TEAM>(s.x + s.y) * inv_e + eps);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < P; ++i) z[r][i] = mul2(z[r][i], pair(inv));
  return inv;
}

// The weight and bias of a thread's channels: kept in registers where they are few.
template <int VEC, int TEAM, int R>
struct Affine {
  static constexpr int P = kPairs<VEC>;
  static constexpr bool kKeep = R * VEC <= 8;
  const float *w, *b;  // of the group
  int chunks;
  float2 wk[kKeep ? R : 1][P], bk[kKeep ? R : 1][P];
  __device__ __forceinline__ Affine(const NormProblem& p, int group, int E, int chunks_) : chunks(chunks_) {
    w = p.w + (size_t)group * E, b = p.bias ? p.bias + (size_t)group * E : nullptr;
    if constexpr (kKeep) {
#pragma unroll
      for (int r = 0; r < R; ++r) fetch(r, wk[r], bk[r]);
    }
  }
  __device__ __forceinline__ void fetch(int r, float2 (&wv)[P], float2 (&bv)[P]) const {
    const int c = Lanes<TEAM>::lane() + r * Lanes<TEAM>::kWidth;
#pragma unroll
    for (int i = 0; i < P; ++i) wv[i] = bv[i] = make_float2(0.f, 0.f);
    if (c >= chunks) return;
    Raw<float, VEC> u;
    u.load(w + (size_t)c * VEC), u.get(wv);
    if (b) u.load(b + (size_t)c * VEC), u.get(bv);
  }
  __device__ __forceinline__ void get(int r, float2 (&wv)[P], float2 (&bv)[P]) const {
    if constexpr (kKeep) {
#pragma unroll
      for (int i = 0; i < P; ++i) wv[i] = wk[r][i], bv[i] = bk[r][i];
    } else {
      fetch(r, wv, bv);
    }
  }
};

// A team takes UNITS groups (rows times groups, `apart`, a multiple of the groups, from one to the
// next), all loaded before the first is computed.
template <typename Y, int VEC, int TEAM, int R, int UNITS, bool GATE>
__global__ void __launch_bounds__(kThreads)
    groupnorm_kernel(NormProblem p, uint16_t* __restrict__ out, int chunks, long long apart) {
  constexpr int P = kPairs<VEC>;
  using L = Lanes<TEAM>;
  const int E = p.D / p.groups;
  const int lane = L::lane();
  const long long first = L::team();
  const int group = (int)(first % p.groups);
  const float inv_e = 1.f / (float)E;
  Raw<Y, VEC> y[UNITS][R];
  Raw<uint16_t, VEC> x[UNITS][R];
  // Unit u starts u * apart * E values after the first: units lie row by row.
  const size_t at = (size_t)first * E, step = (size_t)apart * E;
  bool live[UNITS];
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    live[u] = first < apart && first + u * apart < p.rows * p.groups;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = lane + r * L::kWidth;
      if (live[u] && c < chunks) {
        y[u][r].load(static_cast<const Y*>(p.y) + at + u * step + (size_t)c * VEC);
        if (GATE) x[u][r].load(p.g + at + u * step + (size_t)c * VEC);
      }
    }
  }
  const Affine<VEC, TEAM, R> affine(p, group, E, chunks);
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    float2 z[R][P];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (live[u] && lane + r * L::kWidth < chunks) {
        y[u][r].get(z[r]);
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) z[r][i] = make_float2(0.f, 0.f);
      }
    }
    normalise<VEC, TEAM, R>(live[u], chunks, inv_e, p.eps, z);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = lane + r * L::kWidth;
      if (!live[u] || c >= chunks) break;
      float2 w[P], b[P], o[P], gx[P];
      affine.get(r, w, b);
      if (GATE) x[u][r].get(gx);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        o[i] = fma2(w[i], z[r][i], b[i]);
        o[i] = mul2(o[i], GATE ? mul2(gx[i], sigmoid2(gx[i])) : sigmoid2(o[i]));
      }
      store_vals<VEC>(out + at + u * step + (size_t)c * VEC, o);
    }
  }
}

// Team t of `slots * groups` teams takes group t % groups of rows t / groups, + slots, ...
template <typename Y, int VEC, int TEAM, int R, bool GATE>
__global__ void __launch_bounds__(kThreads)
    groupnorm_backward_kernel(NormProblem p, const uint16_t* __restrict__ dout, Y* __restrict__ dy,
                              uint16_t* __restrict__ dg, float* __restrict__ part, int chunks, int slots) {
  constexpr int P = kPairs<VEC>;
  using L = Lanes<TEAM>;
  const int E = p.D / p.groups;
  const int lane = L::lane();
  const long long t = L::team();
  const int g = (int)(t % p.groups);
  const long long slot = t / p.groups;
  const bool has = slot < slots;
  const float inv_e = 1.f / (float)E;
  const float2 zero = make_float2(0.f, 0.f), one = make_float2(1.f, 1.f);
  float2 dw[R][P], db[R][P];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < P; ++i) dw[r][i] = db[r][i] = zero;
  const Affine<VEC, TEAM, R> affine(p, g, E, chunks);
  const long long steps = (p.rows + slots - 1) / slots;  // the same for every thread
  Raw<Y, VEC> yr[R];
  Raw<uint16_t, VEC> dr[R], xr[R];
  auto load = [&](long long s) {
    const long long row = slot + s * slots;
    if (!has || row >= p.rows) return;
    const size_t at = (size_t)row * p.D + (size_t)g * E;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = lane + r * L::kWidth;
      if (c >= chunks) break;
      yr[r].load(static_cast<const Y*>(p.y) + at + (size_t)c * VEC);
      dr[r].load(dout + at + (size_t)c * VEC);
      if (GATE) xr[r].load(p.g + at + (size_t)c * VEC);
    }
  };
  load(0);
  for (long long s = 0; s < steps; ++s) {
    const long long row = slot + s * slots;
    const bool live = has && row < p.rows;
    const size_t at = live ? (size_t)row * p.D + (size_t)g * E : 0;
    float2 z[R][P], dn[R][P], gx[R][P];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (live && lane + r * L::kWidth < chunks) {
        yr[r].get(z[r]);
        dr[r].get(dn[r]);
        if (GATE) xr[r].get(gx[r]);
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) z[r][i] = dn[r][i] = zero;
      }
    }
    load(s + 1);  // while this row is computed
    const float inv = normalise<VEC, TEAM, R>(live, chunks, inv_e, p.eps, z);
    float2 s1 = zero, s2 = zero;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = lane + r * L::kWidth;
      if (!live || c >= chunks) continue;
      float2 w[P], b[P], o[P];
      affine.get(r, w, b);
#pragma unroll
      for (int i = 0; i < P; ++i) {  // dn becomes dp, then dp w
        const float2 pn = fma2(w[i], z[r][i], b[i]);
        if (GATE) {
          const float2 x = gx[r][i], sig = sigmoid2(x);
          o[i] = mul2(mul2(dn[r][i], pn), mul2(sig, fma2(x, sub2(one, sig), one)));
          dn[r][i] = mul2(dn[r][i], mul2(x, sig));
        } else {
          const float2 sig = sigmoid2(pn);
          dn[r][i] = mul2(dn[r][i], mul2(sig, fma2(pn, sub2(one, sig), one)));
        }
        dw[r][i] = fma2(dn[r][i], z[r][i], dw[r][i]);
        db[r][i] = add2(db[r][i], dn[r][i]);
        dn[r][i] = mul2(dn[r][i], w[i]);
        s1 = add2(s1, dn[r][i]);
        s2 = fma2(dn[r][i], z[r][i], s2);
      }
      if (GATE) store_vals<VEC>(dg + at + (size_t)c * VEC, o);
    }
    const float2 m = team_sum<TEAM>(make_float2(s1.x + s1.y, s2.x + s2.y));
    const float2 m1 = pair(-inv * (m.x * inv_e)), m2 = pair(-inv * (m.y * inv_e)), iv = pair(inv);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = lane + r * L::kWidth;
      if (!live || c >= chunks) break;
      float2 o[P];
#pragma unroll
      for (int i = 0; i < P; ++i) o[i] = fma2(iv, dn[r][i], fma2(z[r][i], m2, m1));
      store_vals<VEC>(dy + at + (size_t)c * VEC, o);
    }
  }
  if (!has) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = lane + r * L::kWidth;
    if (c >= chunks) break;
    float* row = part + (size_t)slot * 2 * p.D + (size_t)g * E + (size_t)c * VEC;
    store_vals<VEC>(row, dw[r]);
    store_vals<VEC>(row + p.D, db[r]);
  }
}

// How a group is spread: lanes per team (0 = the block), chunks of a group, chunks per lane.
struct Shape {
  bool vec;
  int team, chunks, per_lane;
  int width() const { return team ? team : kThreads; }
};

Shape shape_of(int E, bool vec) {
  Shape s{vec, 8, vec ? E / 8 : E, 1};
  while (s.team < 32 && s.team < s.chunks) s.team *= 2;
  s.per_lane = (s.chunks + s.team - 1) / s.team;
  if (s.per_lane > 4) {
    s.team = 0;
    s.per_lane = (s.chunks + kThreads - 1) / kThreads;
  }
  return s;
}

bool vec_ok(const NormProblem& p) {
  return (p.D / p.groups) % 8 == 0 && aligned_to(p.y, 16) && aligned_to(p.g, 16) &&
         aligned_to(p.w, 16) && aligned_to(p.bias, 16);
}

// Rows in flight of the backward: two blocks of teams for every SM, as many as its registers let
// reside (234 us for 131072 rows of 16 x 64 with the sums; four 239, eight 246).
int backward_slots(long long rows, int D, int groups) {
  const Shape s = shape_of(D / groups, (D / groups) % 8 == 0);
  long long teams = 152LL * 2 * (kThreads / s.width());
  long long slots = teams / groups;
  if (slots < 1) slots = 1;
  return (int)(slots < rows ? slots : rows > 0 ? rows : 1);
}

// Calls f with the kernel's compile-time shape: f(vec constant, team constant, values constant).
template <int N>
struct Int {
  static constexpr int value = N;
};
template <typename F>
cudaError_t with_shape(const Shape& s, F f) {
  if (s.vec) {
    if (s.team == 8) return f(Int<8>{}, Int<8>{}, Int<1>{});
    if (s.team == 16) return f(Int<8>{}, Int<16>{}, Int<1>{});
    if (s.team == 32) {
      if (s.per_lane == 1) return f(Int<8>{}, Int<32>{}, Int<1>{});
      if (s.per_lane == 2) return f(Int<8>{}, Int<32>{}, Int<2>{});
      return f(Int<8>{}, Int<32>{}, Int<4>{});
    }
    if (s.per_lane <= 2) return f(Int<8>{}, Int<0>{}, Int<2>{});
    return f(Int<8>{}, Int<0>{}, Int<4>{});
  }
  if (s.team == 8) return f(Int<1>{}, Int<8>{}, Int<1>{});
  if (s.team == 16) return f(Int<1>{}, Int<16>{}, Int<1>{});
  if (s.team == 32) return f(Int<1>{}, Int<32>{}, Int<4>{});
  if (s.per_lane <= 4) return f(Int<1>{}, Int<0>{}, Int<4>{});
  return f(Int<1>{}, Int<0>{}, Int<32>{});
}

template <typename Y, bool GATE>
cudaError_t forward_typed(const NormProblem& p, uint16_t* out, const Shape& s, cudaStream_t stream) {
  const long long units = p.rows * p.groups, per_block = kThreads / s.width();
  return with_shape(s, [&](auto vec, auto team, auto r) {
    constexpr int V = decltype(vec)::value, G = decltype(team)::value, R = decltype(r)::value;
    // Three units per team where that still fills the GPU (131072 rows of 16 x 64: 136 us; by two 140, by
    // one 164).
    constexpr int U = R * V == 8 ? 3 : 1;
    const bool many = U > 1 && units >= 152LL * 4 * per_block * U;
    const long long apart = many ? ((p.rows + U - 1) / U) * p.groups : units;
    const unsigned blocks = (unsigned)((apart + per_block - 1) / per_block);
    if (many)
      groupnorm_kernel<Y, V, G, R, U, GATE><<<blocks, kThreads, 0, stream>>>(p, out, s.chunks, apart);
    else
      groupnorm_kernel<Y, V, G, R, 1, GATE><<<blocks, kThreads, 0, stream>>>(p, out, s.chunks, apart);
    return cudaGetLastError();
  });
}

template <typename Y, bool GATE>
cudaError_t backward_typed(const NormProblem& p, const uint16_t* dout, void* dy, uint16_t* dg,
                           float* part, int slots, const Shape& s, cudaStream_t stream) {
  const long long teams = (long long)slots * p.groups, per_block = kThreads / s.width();
  const unsigned blocks = (unsigned)((teams + per_block - 1) / per_block);
  return with_shape(s, [&](auto vec, auto team, auto r) {
    groupnorm_backward_kernel<Y, decltype(vec)::value, decltype(team)::value, decltype(r)::value, GATE>
        <<<blocks, kThreads, 0, stream>>>(p, dout, static_cast<Y*>(dy), dg, part, s.chunks, slots);
    return cudaGetLastError();
  });
}

// Calls f with the type of y and whether there is a gate.
template <typename F>
cudaError_t with_kind(const NormProblem& p, F f) {
  if (p.y_f32) return p.g ? f(0.f, Int<1>{}) : f(0.f, Int<0>{});
  return p.g ? f(uint16_t{}, Int<1>{}) : f(uint16_t{}, Int<0>{});
}

}  // namespace

cudaError_t launch_groupnorm(const NormProblem& p, uint16_t* out, cudaStream_t stream) {
  const Shape s = shape_of(p.D / p.groups, vec_ok(p) && aligned_to(out, 16));
  return with_kind(p, [&](auto y, auto gate) {
    return forward_typed<decltype(y), decltype(gate)::value != 0>(p, out, s, stream);
  });
}

// Partial rows [slots][dw, db][D].
size_t groupnorm_backward_workspace_floats(long long rows, int D, int groups) {
  return (size_t)backward_slots(rows, D, groups) * 2 * D;
}

cudaError_t launch_groupnorm_backward(const NormProblem& p, const uint16_t* dout, void* dy,
                                      uint16_t* dg, float* dw, float* dbias, float* ws,
                                      cudaStream_t stream) {
  if (p.rows == 0) {
    cudaError_t err = cudaMemsetAsync(dw, 0, sizeof(float) * p.D, stream);
    if (err == cudaSuccess && dbias) err = cudaMemsetAsync(dbias, 0, sizeof(float) * p.D, stream);
    return err;
  }
  const Shape s = shape_of(p.D / p.groups, vec_ok(p) && aligned_to(dout, 16) && aligned_to(dy, 16) &&
                                               aligned_to(dg, 16));
  const int slots = backward_slots(p.rows, p.D, p.groups);
  const cudaError_t err = with_kind(p, [&](auto y, auto gate) {
    return backward_typed<decltype(y), decltype(gate)::value != 0>(p, dout, dy, dg, ws, slots, s, stream);
  });
  if (err != cudaSuccess) return err;
  return launch_sum_rows(ws, dw, dbias, slots, p.D, dbias ? 2 * p.D : p.D,
                         2 * p.D, stream);
}

}  // namespace m2rnn
