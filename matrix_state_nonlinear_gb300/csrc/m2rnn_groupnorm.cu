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

// The group's values in registers, centred and scaled: z = n; returns inv.
template <typename Y, int VEC, bool BLOCK, int R>
__device__ __forceinline__ float load_normalised(const Y* y, bool live, int lane, int team, int chunks,
                                                 int E, float eps, float (&z)[R][VEC]) {
  float s = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = lane + r * team;
    if (live && c < chunks) {
      load_vals<VEC>(y + (size_t)c * VEC, z[r]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) z[r][i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) s += z[r][i];
  }
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

template <typename Y, int VEC, bool BLOCK, int R>
__global__ void __launch_bounds__(kThreads)
    groupnorm_kernel(NormProblem p, uint16_t* __restrict__ out, int team, int chunks) {
  const int E = p.D / p.groups;
  const int lane = BLOCK ? threadIdx.x : threadIdx.x & (team - 1);
  const long long unit = BLOCK ? blockIdx.x
                               : ((long long)blockIdx.x * kThreads + threadIdx.x) / team;
  const bool live = unit < p.rows * p.groups;
  const int g = (int)(unit % p.groups);
  const size_t at = live ? (size_t)(unit / p.groups) * p.D + (size_t)g * E : 0;
  float z[R][VEC];
  load_normalised<Y, VEC, BLOCK, R>(static_cast<const Y*>(p.y) + at, live, lane, team, chunks, E,
                                    p.eps, z);
  if (!live) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = lane + r * team;
    if (c >= chunks) break;
    const size_t e = (size_t)c * VEC;
    float w[VEC], b[VEC], o[VEC];
    load_vals<VEC>(p.w + (size_t)g * E + e, w);
    if (p.bias) load_vals<VEC>(p.bias + (size_t)g * E + e, b);
#pragma unroll
    for (int i = 0; i < VEC; ++i) o[i] = fmaf(w[i], z[r][i], p.bias ? b[i] : 0.f);
    if (p.g) {
      float x[VEC];
      load_vals<VEC>(p.g + at + e, x);
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] *= x[i] * sigmoid_f(x[i]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] *= sigmoid_f(o[i]);
    }
    store_vals<VEC>(out + at + e, o);
  }
}

// Team t of `slots * groups` teams takes group t % groups of rows t / groups, + slots, ...
template <typename Y, int VEC, bool BLOCK, int R>
__global__ void __launch_bounds__(kThreads)
    groupnorm_backward_kernel(NormProblem p, const uint16_t* __restrict__ dout, Y* __restrict__ dy,
                              uint16_t* __restrict__ dg, float* __restrict__ part, int team,
                              int chunks, int slots) {
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
  for (long long s = 0; s < steps; ++s) {
    const long long row = slot + s * slots;
    const bool live = has && row < p.rows;
    const size_t at = live ? (size_t)row * p.D + (size_t)g * E : 0;
    float z[R][VEC], dn[R][VEC];
    const float inv = load_normalised<Y, VEC, BLOCK, R>(static_cast<const Y*>(p.y) + at, live, lane,
                                                        team, chunks, E, p.eps, z);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = lane + r * team;
      if (!live || c >= chunks) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) dn[r][i] = 0.f;
        continue;
      }
      const size_t e = (size_t)c * VEC;
      float w[VEC], b[VEC], d[VEC];
      load_vals<VEC>(p.w + (size_t)g * E + e, w);
      if (p.bias) load_vals<VEC>(p.bias + (size_t)g * E + e, b);
      load_vals<VEC>(dout + at + e, d);
      if (p.g) {
        float x[VEC], o[VEC];
        load_vals<VEC>(p.g + at + e, x);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float sig = sigmoid_f(x[i]);
          const float pn = fmaf(w[i], z[r][i], p.bias ? b[i] : 0.f);
          o[i] = d[i] * pn * (sig * fmaf(x[i], 1.f - sig, 1.f));
          dn[r][i] = d[i] * (x[i] * sig);
        }
        store_vals<VEC>(dg + at + e, o);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float pn = fmaf(w[i], z[r][i], p.bias ? b[i] : 0.f);
          const float sig = sigmoid_f(pn);
          dn[r][i] = d[i] * (sig * fmaf(pn, 1.f - sig, 1.f));
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
  long long teams = 152LL * 6 * (s.block ? 1 : kThreads / s.team);
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
  const unsigned blocks = (unsigned)((units + per_block - 1) / per_block);
  return with_shape(s, [&](auto vec, auto block, auto r) {
    groupnorm_kernel<Y, decltype(vec)::value, decltype(block)::value != 0, decltype(r)::value>
        <<<blocks, kThreads, 0, stream>>>(p, out, s.team, s.chunks);
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
