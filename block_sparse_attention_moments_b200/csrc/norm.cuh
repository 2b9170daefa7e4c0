// norm.cuh — norms before and after a block, with modulation, gate, residual
// and quantisation, one pass over the rows.
//
// For a token's row x of C channels, and y, the output of the block before:
//   x' = rs * x + gate * post(y)            (without y: x' = x)
//   h  = pre(x') * (1 + scale) + shift
// pre and post are
//   layer  (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps) * weight + bias
//   rms    v / sqrt(mean(v^2) + eps) * weight + bias
//   none   v
// and h is written as it is, or in 8 bits with a scale for the row:
//   s = max|h| / 127,  q = round(h / s)
//
// Everything between the loads and the stores is fp32 in registers: the row is
// read once, the variance is the mean square of the centred values (no
// difference of large sums), and h comes from the x' before its rounding.
// The parts that multiply and add along the channels are folded:
//   h = n * A + B   with A = weight * (1 + scale),  B = bias * (1 + scale) + shift
//   x' = rs * x + n_y * PA + PB  with PA = gate * post_weight, PB = gate * post_bias
#pragma once

#include "rows.cuh"

namespace solattn {

enum : int { kNormNone = 0, kNormLayer = 1, kNormRms = 2 };

// [B, G, C]: group g covers `per` consecutive tokens.  p is null where absent.
struct Vectors {
  const void* p;
  long long sb, sg;
  int dtype;
  int per;
};

struct NormParams {
  int B, L, C;
  // x, y: channel c of token (b, l) lies at b*sb + l*sl + (c / inner)*sh + c % inner
  const void* x;
  long long x_sb, x_sl, x_sh;
  int x_inner;
  const void* y;
  long long y_sb, y_sl;
  void* xo;                       // x' (null: not wanted)
  long long xo_sb, xo_sl;
  void* h;                        // h in the type of y (null: not wanted)
  long long h_sb, h_sl;
  int8_t* q;                      // h in 8 bits (null: not wanted), row pitch q_sl
  long long q_sl;
  float* q_scale;                 // [B * L]
  float rs;
  int pre, post;
  float pre_eps, post_eps;
  Vectors scale, shift, gate, weight, bias, post_weight, post_bias;
  int warps;                      // warps of a team
};

template <int V>
__device__ __forceinline__ bool load_vectors(const Vectors& v, int b, int l, int c, float (&f)[V]) {
  if (!v.p) return false;
  load_param<V>(v.p, v.dtype, b * v.sb + (l / v.per) * v.sg + c, f);
  return true;
}

template <int V>
__device__ __forceinline__ void fold_pre(const NormParams& p, int b, int l, int c, float (&A)[V], float (&Bv)[V]) {
  float t[V];
#pragma unroll
  for (int j = 0; j < V; ++j) A[j] = 1.f, Bv[j] = 0.f;
  if (load_vectors<V>(p.weight, b, l, c, t)) {
#pragma unroll
    for (int j = 0; j < V; ++j) A[j] = t[j];
  }
  load_vectors<V>(p.bias, b, l, c, Bv);
  if (load_vectors<V>(p.scale, b, l, c, t)) {
#pragma unroll
    for (int j = 0; j < V; ++j) A[j] *= 1.f + t[j], Bv[j] *= 1.f + t[j];
  }
  if (load_vectors<V>(p.shift, b, l, c, t)) {
#pragma unroll
    for (int j = 0; j < V; ++j) Bv[j] += t[j];
  }
}

template <int V>
__device__ __forceinline__ void fold_post(const NormParams& p, int b, int l, int c, float (&A)[V], float (&Bv)[V]) {
  float t[V];
#pragma unroll
  for (int j = 0; j < V; ++j) A[j] = 1.f, Bv[j] = 0.f;
  if (load_vectors<V>(p.post_weight, b, l, c, t)) {
#pragma unroll
    for (int j = 0; j < V; ++j) A[j] = t[j];
  }
  load_vectors<V>(p.post_bias, b, l, c, Bv);
  if (load_vectors<V>(p.gate, b, l, c, t)) {
#pragma unroll
    for (int j = 0; j < V; ++j) A[j] *= t[j], Bv[j] *= t[j];
  }
}

// Normalises a row that the team holds in registers (no weight or bias).
template <int V, int N>
__device__ __forceinline__ void normalise(Team& t, int kind, float eps, int C, const bool (&on)[N], float (&v)[N][V]) {
  if (kind == kNormNone) return;
  const float n = static_cast<float>(C);
  if (kind == kNormLayer) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) s += v[i][j];   // zero outside the row
    const float mean = team_sum(t, s) / n;   // a division: the mean of equal values is that value
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = on[i] ? v[i][j] - mean : 0.f;
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) s = fmaf(v[i][j], v[i][j], s);
  const float r = rsqrtf(team_sum(t, s) / n + eps);
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) v[i][j] *= r;
}

constexpr int kNormThreads = 512;

// One team to a row; thread t of the team holds the row's vectors t, t + T,
// t + 2T, ... (T threads, N vectors of V elements at most).
template <typename TX, typename TY, int V, int N, bool RES>
__global__ void __launch_bounds__(kNormThreads, 1) norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float slots[2 * (kNormThreads / 32)];
  Team team;
  team.warps = p.warps;
  team.index = (threadIdx.x / 32) / p.warps;
  team.warp = (threadIdx.x / 32) % p.warps;
  team.slots = slots + 2 * p.warps * team.index;
  team.turn = 0;
  const int teams = blockDim.x / 32 / p.warps;
  const int T = p.warps * 32;
  const int tid = threadIdx.x - team.index * T;
  const int nvec = p.C / V;
  const long long rows = static_cast<long long>(p.B) * p.L;

  bool on[N];
#pragma unroll
  for (int i = 0; i < N; ++i) on[i] = tid + i * T < nvec;

  for (long long row = static_cast<long long>(blockIdx.x) * teams + team.index; row < rows;
       row += static_cast<long long>(gridDim.x) * teams) {
    const int b = static_cast<int>(row / p.L);
    const int l = static_cast<int>(row - static_cast<long long>(b) * p.L);

    Raw<TX, V> rx[N];
    Raw<TY, V> ry[N];
    const TX* xp = static_cast<const TX*>(p.x) + b * p.x_sb + l * p.x_sl;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!on[i]) continue;
      const int c = (tid + i * T) * V;
      load_raw(rx[i], xp + (p.x_inner == p.C ? c : (c / p.x_inner) * p.x_sh + c % p.x_inner));
    }
    if constexpr (RES) {
      const TY* yp = static_cast<const TY*>(p.y) + b * p.y_sb + l * p.y_sl;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (on[i]) load_raw(ry[i], yp + (tid + i * T) * V);
    }

    float v[N][V];
    if constexpr (RES) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (on[i]) widen(ry[i], v[i]);
        else
#pragma unroll
          for (int j = 0; j < V; ++j) v[i][j] = 0.f;
      }
      normalise<V, N>(team, p.post, p.post_eps, p.C, on, v);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (!on[i]) continue;
        float A[V], Bv[V], x[V];
        fold_post<V>(p, b, l, (tid + i * T) * V, A, Bv);
        widen(rx[i], x);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] = fmaf(p.rs, x[j], fmaf(v[i][j], A[j], Bv[j]));
      }
      if (p.xo) {
        TX* op = static_cast<TX*>(p.xo) + b * p.xo_sb + l * p.xo_sl;
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (on[i]) store_row(op + (tid + i * T) * V, v[i]);
      }
      if (!p.h && !p.q) continue;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (!on[i])
#pragma unroll
          for (int j = 0; j < V; ++j) v[i][j] = 0.f;
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (on[i]) widen(rx[i], v[i]);
        else
#pragma unroll
          for (int j = 0; j < V; ++j) v[i][j] = 0.f;
      }
    }

    normalise<V, N>(team, p.pre, p.pre_eps, p.C, on, v);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!on[i]) continue;
      float A[V], Bv[V];
      fold_pre<V>(p, b, l, (tid + i * T) * V, A, Bv);
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = fmaf(v[i][j], A[j], Bv[j]);
    }
    if (p.h) {
      TY* hp = static_cast<TY*>(p.h) + b * p.h_sb + l * p.h_sl;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (on[i]) store_row(hp + (tid + i * T) * V, v[i]);
    }
    if (p.q) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (on[i]) m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
      const float amax = __uint_as_float(team_max(team, m));
      // a row of zeros: scale 0 and zeros; a row with an infinity or a NaN:
      // a scale that is not finite and zeros, so that what is made of it is NaN
      const bool plain = amax > 0.f && amax <= 3.402823466e38f;
      // h / s as h * (127 / amax) (an amax below 127 / FLT_MAX would overflow
      // the quotient; there the division itself is taken)
      const float up = 127.f / amax;
      const float s = amax / 127.f;
      const bool tiny = plain && !(up <= 3.402823466e38f);
      int8_t* qp = p.q + row * p.q_sl;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (!on[i]) continue;
        int k[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float u = tiny ? (v[i][j] / amax) * 127.f : v[i][j] * up;
          k[j] = plain ? max(-127, min(127, __float2int_rn(u))) : 0;
        }
        if constexpr (V == 8) {
          uint2 w;
          w.x = (k[0] & 255) | (k[1] & 255) << 8 | (k[2] & 255) << 16 | static_cast<uint32_t>(k[3]) << 24;
          w.y = (k[4] & 255) | (k[5] & 255) << 8 | (k[6] & 255) << 16 | static_cast<uint32_t>(k[7]) << 24;
          *reinterpret_cast<uint2*>(qp + (tid + i * T) * 8) = w;
        } else {
          qp[tid + i * T] = static_cast<int8_t>(k[0]);
        }
      }
      if (tid == 0) p.q_scale[row] = s;
    }
  }
}

}  // namespace solattn
