// m2rnn_groupnorm.cu — gated group norm over the channels of one token, and its backward.
//
//   n = (y - mean) inv,  inv = 1 / sqrt(var + eps),  p = w n + b
//   out = p s(g)  (s = SiLU, with a gate)   or   out = s(p)  (without)
// Backward, with dp = dout s(g) or dout s'(p):
//   dg = dout p s'(g),  dw = sum dp n,  db = sum dp,  dn = dp w
//   dy = inv (dn - mean(dn) - n mean(dn n))
//
// Memory-bound.  A team of lanes takes one group of one row: each lane holds its share in
// registers, so y is read once, and mean and variance are two exact passes over registers (the
// variance of the centred values; no sum of squares is subtracted).  A team is 1 to 32 lanes of
// a warp, or the whole block for groups of more than 32 lanes' registers.  The backward keeps
// a team on the same channels for many rows, so that dw and db add up in registers, and one
// row of partial sums per team goes to memory.
#include "m2rnn_ssm.h"
#include "ptx_util.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// VEC values as loaded, so that a load can be started ahead of its use.
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
  __device__ __forceinline__ void get(float (&f)[VEC]) const {
    if constexpr (VEC == 8 && sizeof(Y) == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(u[i].x), f[4 * i + 1] = __uint_as_float(u[i].y);
        f[4 * i + 2] = __uint_as_float(u[i].z), f[4 * i + 3] = __uint_as_float(u[i].w);
      }
    } else if constexpr (VEC == 8) {
      f[0] = bf16_lo(u[0].x), f[1] = bf16_hi(u[0].x), f[2] = bf16_lo(u[0].y), f[3] = bf16_hi(u[0].y);
      f[4] = bf16_lo(u[0].z), f[5] = bf16_hi(u[0].z), f[6] = bf16_lo(u[0].w), f[7] = bf16_hi(u[0].w);
    } else {
      f[0] = sizeof(Y) == 4 ? __uint_as_float(u[0].x) : bf16_to_f((uint16_t)u[0].x);
    }
  }
};

// VEC values at p, as floats.
template <int VEC>
__device__ __forceinline__ void load_vals(const uint16_t* p, float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    f[0] = bf16_lo(u.x), f[1] = bf16_hi(u.x), f[2] = bf16_lo(u.y), f[3] = bf16_hi(u.y);
    f[4] = bf16_lo(u.z), f[5] = bf16_hi(u.z), f[6] = bf16_lo(u.w), f[7] = bf16_hi(u.w);
  } else {
    f[0] = bf16_to_f(*p);
  }
}
template <int VEC>
__device__ __forceinline__ void load_vals(const float* p, float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    f[0] = *p;
  }
}
template <int VEC>
__device__ __forceinline__ void store_vals(uint16_t* p, const float (&f)[VEC]) {
  if constexpr (VEC == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                              pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  else
    *p = f_to_bf16(f[0]);
}
template <int VEC>
__device__ __forceinline__ void store_vals(float* p, const float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *p = f[0];
  }
}

// Sum over the team: `team` lanes of a warp (a power of two), or the whole block.  Every thread
// of the block calls it (lanes without a group pass zeros).
template <bool BLOCK>
__device__ __forceinline__ float team_sum(float s, int team) {
  if constexpr (!BLOCK) {
    for (int o = team / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  } else {
    __shared__ float part[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += part[w];
    __syncthreads();
    return s;
  }
}

// Centres and scales a group's values (zeros outside it): z becomes n; returns inv.
template <int VEC, bool BLOCK, int R>
__device__ __forceinline__ float normalise(bool live, int lane, int team, int chunks, int E, float eps,
                                           float (&z)[R][VEC]) {
  float s = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < VEC; ++i) s += z[r][i];
  const float mean = team_sum<BLOCK>(s, team) / (float)E;
  s = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const bool in = live && lane + r * team < chunks;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      z[r][i] = in ? z[r][i] - mean : 0.f;
      s = fmaf(z[r][i], z[r][i], s);
    }
  }
  const float inv = rsqrtf(team_sum<BLOCK>(s, team) / (float)E + eps);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < VEC; ++i) z[r][i] *= inv;
  return inv;
}

// A team takes UNITS groups, `apart` units from one to the next, all loaded before the first is
// computed.
template <typename Y, int VEC, bool BLOCK, int R, int UNITS>
__global__ void __launch_bounds__(kThreads)
    groupnorm_kernel(NormProblem p, uint16_t* __restrict__ out, int team, int chunks, long long apart) {
  const int E = p.D / p.groups;
  const int lane = BLOCK ? threadIdx.x : threadIdx.x & (team - 1);
  const long long first = BLOCK ? blockIdx.x
                                : ((long long)blockIdx.x * kThreads + threadIdx.x) / team;
  Raw<Y, VEC> y[UNITS][R];
  Raw<uint16_t, VEC> x[UNITS][R];
  size_t at[UNITS];
  bool live[UNITS];
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const long long unit = first + u * apart;
    live[u] = first < apart && unit < p.rows * p.groups;
    at[u] = live[u] ? (size_t)(unit / p.groups) * p.D + (size_t)(unit % p.groups) * E : 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = lane + r * team;
      if (live[u] && c < chunks) {
        y[u][r].load(static_cast<const Y*>(p.y) + at[u] + (size_t)c * VEC);
        if (p.g) x[u][r].load(p.g + at[u] + (size_t)c * VEC);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int g = (int)((first + u * apart) % p.groups);
    float z[R][VEC];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (live[u] && lane + r * team < chunks) {
        y[u][r].get(z[r]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) z[r][i] = 0.f;
      }
    }
    normalise<VEC, BLOCK, R>(live[u], lane, team, chunks, E, p.eps, z);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = lane + r * team;
      if (!live[u] || c >= chunks) break;
      const size_t e = (size_t)c * VEC;
      float w[VEC], b[VEC], o[VEC];
      load_vals<VEC>(p.w + (size_t)g * E + e, w);
      if (p.bias) load_vals<VEC>(p.bias + (size_t)g * E + e, b);
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] = fmaf(w[i], z[r][i], p.bias ? b[i] : 0.f);
      if (p.g) {
        float gx[VEC];
        x[u][r].get(gx);
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] *= gx[i] * sigmoid_f(gx[i]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] *= sigmoid_f(o[i]);
      }
      store_vals<VEC>(out + at[u] + e, o);
    }
  }
}

// Team t of `slots * groups` teams takes group t % groups of rows t / groups, + slots, ...; the next
// row is loaded while one is computed.
template <typename Y, int VEC, bool BLOCK, int R>
__global__ void __launch_bounds__(kThreads)
    groupnorm_backward_kernel(NormProblem p, const uint16_t* __restrict__ dout, Y* __restrict__ dy,
                              uint16_t* __restrict__ dg, float* __restrict__ part, int team,
                              int chunks, int slots) {
  constexpr bool kAhead = R * VEC <= 16;  // as far as registers go
  const int E = p.D / p.groups;
  const int lane = BLOCK ? threadIdx.x : threadIdx.x & (team - 1);
  const long long t = BLOCK ? blockIdx.x
                            : ((long long)blockIdx.x * kThreads + threadIdx.x) / team;
  const int g = (int)(t % p.groups);
  const long long slot = t / p.groups;
  const bool has = slot < slots;
  float dw[R][VEC], db[R][VEC];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < VEC; ++i) dw[r][i] = db[r][i] = 0.f;
  const long long steps = (p.rows + slots - 1) / slots;  // the same for every thread
  Raw<Y, VEC> yr[R];
  Raw<uint16_t, VEC> dr[R], xr[R];
  auto load = [&](long long s) {
    const long long row = slot + s * slots;
    if (!has || row >= p.rows) return;
    const size_t at = (size_t)row * p.D + (size_t)g * E;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = lane + r * team;
      if (c >= chunks) break;
      yr[r].load(static_cast<const Y*>(p.y) + at + (size_t)c * VEC);
      dr[r].load(dout + at + (size_t)c * VEC);
      if (p.g) xr[r].load(p.g + at + (size_t)c * VEC);
    }
  };
  if (kAhead) load(0);
  for (long long s = 0; s < steps; ++s) {
    const long long row = slot + s * slots;
    const bool live = has && row < p.rows;
    const size_t at = live ? (size_t)row * p.D + (size_t)g * E : 0;
    if (!kAhead) load(s);
    float z[R][VEC], dn[R][VEC], gx[kAhead ? R : 1][VEC];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (live && lane + r * team < chunks) {
        yr[r].get(z[r]);
        dr[r].get(dn[r]);
        if (kAhead && p.g) xr[r].get(gx[kAhead ? r : 0]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) z[r][i] = dn[r][i] = 0.f;
      }
    }
    if (kAhead) load(s + 1);
    const float inv = normalise<VEC, BLOCK, R>(live, lane, team, chunks, E, p.eps, z);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = lane + r * team;
      if (!live || c >= chunks) continue;
      const size_t e = (size_t)c * VEC;
      float w[VEC], b[VEC], x[VEC];
      load_vals<VEC>(p.w + (size_t)g * E + e, w);
      if (p.bias) load_vals<VEC>(p.bias + (size_t)g * E + e, b);
      if (p.g) {
        if (!kAhead) xr[r].get(x);
        float o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float xi = kAhead ? gx[kAhead ? r : 0][i] : x[i];
          const float sig = sigmoid_f(xi);
          const float pn = fmaf(w[i], z[r][i], p.bias ? b[i] : 0.f);
          o[i] = dn[r][i] * pn * (sig * fmaf(xi, 1.f - sig, 1.f));
          dn[r][i] *= xi * sig;
        }
        store_vals<VEC>(dg + at + e, o);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float pn = fmaf(w[i], z[r][i], p.bias ? b[i] : 0.f);
          const float sig = sigmoid_f(pn);
          dn[r][i] *= sig * fmaf(pn, 1.f - sig, 1.f);
        }
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) {  // dn holds dp here
        dw[r][i] = fmaf(dn[r][i], z[r][i], dw[r][i]);
        db[r][i] += dn[r][i];
        dn[r][i] *= w[i];
        s1 += dn[r][i];
        s2 = fmaf(dn[r][i], z[r][i], s2);
      }
    }
    const float m1 = team_sum<BLOCK>(s1, team) / (float)E;
    const float m2 = team_sum<BLOCK>(s2, team) / (float)E;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = lane + r * team;
      if (!live || c >= chunks) break;
      float o[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] = inv * (dn[r][i] - m1 - z[r][i] * m2);
      store_vals<VEC>(dy + at + (size_t)c * VEC, o);
    }
  }
  if (!has) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = lane + r * team;
    if (c >= chunks) break;
    float* row = part + (size_t)slot * 2 * p.D + (size_t)g * E + (size_t)c * VEC;
    store_vals<VEC>(row, dw[r]);
    store_vals<VEC>(row + p.D, db[r]);
  }
}

// How a group is spread: lanes per team and values per lane.
struct Shape {
  bool vec, block;
  int team, chunks, per_lane;
};
Shape shape_of(int E, bool vec) {
  Shape s{vec, false, 1, vec ? E / 8 : E, 1};
  while (s.team < 32 && s.team < s.chunks) s.team *= 2;
  s.per_lane = (s.chunks + s.team - 1) / s.team;
  if (s.per_lane > 4) {
    s.block = true;
    s.team = kThreads;
    s.per_lane = (s.chunks + s.team - 1) / s.team;
  }
  return s;
}

bool vec_ok(const NormProblem& p) {
  return (p.D / p.groups) % 8 == 0 && aligned_to(p.y, 16) && aligned_to(p.g, 16) &&
         aligned_to(p.w, 16) && aligned_to(p.bias, 16);
}

// Rows in flight of the backward: enough teams for every SM, few enough partial sums.
int backward_slots(long long rows, int D, int groups) {
  const Shape s = shape_of(D / groups, (D / groups) % 8 == 0);
  long long teams = 152LL * 4 * (s.block ? 1 : kThreads / s.team);
  long long slots = teams / groups;
  if (slots < 1) slots = 1;
  return (int)(slots < rows ? slots : rows > 0 ? rows : 1);
}

// Calls f with the kernel's compile-time shape: f(vec constant, block constant, values constant).
template <int N>
struct Int {
  static constexpr int value = N;
};
template <typename F>
cudaError_t with_shape(const Shape& s, F f) {
  if (s.vec) {
    if (!s.block) {
      if (s.per_lane == 1) return f(Int<8>{}, Int<0>{}, Int<1>{});
      if (s.per_lane == 2) return f(Int<8>{}, Int<0>{}, Int<2>{});
      return f(Int<8>{}, Int<0>{}, Int<4>{});
    }
    if (s.per_lane <= 2) return f(Int<8>{}, Int<1>{}, Int<2>{});
    return f(Int<8>{}, Int<1>{}, Int<4>{});
  }
  if (!s.block) {
    if (s.per_lane == 1) return f(Int<1>{}, Int<0>{}, Int<1>{});
    return f(Int<1>{}, Int<0>{}, Int<4>{});
  }
  if (s.per_lane <= 4) return f(Int<1>{}, Int<1>{}, Int<4>{});
  return f(Int<1>{}, Int<1>{}, Int<32>{});
}

template <typename Y>
cudaError_t forward_typed(const NormProblem& p, uint16_t* out, const Shape& s, cudaStream_t stream) {
  const long long units = p.rows * p.groups;
  const long long per_block = s.block ? 1 : kThreads / s.team;
  return with_shape(s, [&](auto vec, auto block, auto r) {
    constexpr int V = decltype(vec)::value, R = decltype(r)::value;
    constexpr bool B = decltype(block)::value != 0;
    // Several units per team where there are enough of them to fill the GPU all the same.
    constexpr int U = R * V <= 8 ? 4 : R * V <= 16 ? 2 : 1;
    if (U > 1 && units >= 152LL * 8 * per_block * U) {
      const long long apart = (units + U - 1) / U;
      groupnorm_kernel<Y, V, B, R, U>
          <<<(unsigned)((apart + per_block - 1) / per_block), kThreads, 0, stream>>>(p, out, s.team, s.chunks, apart);
    } else {
      groupnorm_kernel<Y, V, B, R, 1>
          <<<(unsigned)((units + per_block - 1) / per_block), kThreads, 0, stream>>>(p, out, s.team, s.chunks, units);
    }
    return cudaGetLastError();
  });
}

template <typename Y>
cudaError_t backward_typed(const NormProblem& p, const uint16_t* dout, void* dy, uint16_t* dg,
                           float* part, int slots, const Shape& s, cudaStream_t stream) {
  const long long teams = (long long)slots * p.groups;
  const long long per_block = s.block ? 1 : kThreads / s.team;
  const unsigned blocks = (unsigned)((teams + per_block - 1) / per_block);
  return with_shape(s, [&](auto vec, auto block, auto r) {
    groupnorm_backward_kernel<Y, decltype(vec)::value, decltype(block)::value != 0,
                              decltype(r)::value><<<blocks, kThreads, 0, stream>>>(
        p, dout, static_cast<Y*>(dy), dg, part, s.team, s.chunks, slots);
    return cudaGetLastError();
  });
}

}  // namespace

cudaError_t launch_groupnorm(const NormProblem& p, uint16_t* out, cudaStream_t stream) {
  const Shape s = shape_of(p.D / p.groups, vec_ok(p) && aligned_to(out, 16));
  return p.y_f32 ? forward_typed<float>(p, out, s, stream)
                 : forward_typed<uint16_t>(p, out, s, stream);
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
  const cudaError_t err =
      p.y_f32 ? backward_typed<float>(p, dout, dy, dg, ws, slots, s, stream)
              : backward_typed<uint16_t>(p, dout, dy, dg, ws, slots, s, stream);
  if (err != cudaSuccess) return err;
  return launch_sum_rows(ws, dw, dbias, slots, p.D, dbias ? 2 * p.D : p.D,
                         2 * p.D, stream);
}

}  // namespace m2rnn
