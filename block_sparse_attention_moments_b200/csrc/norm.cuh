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
  int group;                      // tokens that share all of their vectors
};

// The folded factors of N vectors of V channels, c, c + step, ...
template <int V, int N>
__device__ __forceinline__ void apply(const Vectors& v, int b, int l, int c, int step, int end, float (&t)[N][V]) {
  load_params<V, N>(v.p, v.dtype, b * v.sb + (l / v.per) * v.sg, c, step, end, t);
}
template <int V, int N>
__device__ __forceinline__ void fold_pre(const NormParams& p, int b, int l, int c, int step, float (&A)[N][V],
                                         float (&Bv)[N][V]) {
  float t[N][V];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) A[i][j] = 1.f, Bv[i][j] = 0.f, t[i][j] = 0.f;
  if (p.weight.p) apply<V, N>(p.weight, b, l, c, step, p.C, A);
  if (p.bias.p) apply<V, N>(p.bias, b, l, c, step, p.C, Bv);
  if (p.scale.p) {
    apply<V, N>(p.scale, b, l, c, step, p.C, t);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) A[i][j] *= 1.f + t[i][j], Bv[i][j] *= 1.f + t[i][j];
  }
  if (p.shift.p) {
    apply<V, N>(p.shift, b, l, c, step, p.C, t);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) Bv[i][j] += t[i][j];
  }
}
template <int V, int N>
__device__ __forceinline__ void fold_post(const NormParams& p, int b, int l, int c, int step, float (&A)[N][V],
                                          float (&Bv)[N][V]) {
  float t[N][V];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) A[i][j] = 1.f, Bv[i][j] = 0.f, t[i][j] = 0.f;
  if (p.post_weight.p) apply<V, N>(p.post_weight, b, l, c, step, p.C, A);
  if (p.post_bias.p) apply<V, N>(p.post_bias, b, l, c, step, p.C, Bv);
  if (p.gate.p) {
    apply<V, N>(p.gate, b, l, c, step, p.C, t);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) A[i][j] *= t[i][j], Bv[i][j] *= t[i][j];
  }
}

// Factors in shared memory: a plane of the first four channels of each vector
// and one of the last four, so that a warp's 16-byte accesses have no conflicts.
template <int V>
__device__ __forceinline__ void put_factor(float* plane, int nvec, int vec, const float (&f)[V]) {
  if constexpr (V == 8) {
    reinterpret_cast<float4*>(plane)[vec] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(plane)[nvec + vec] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    plane[vec] = f[0];
  }
}
template <int V>
__device__ __forceinline__ void get_factor(const float* plane, int nvec, int vec, float (&f)[V]) {
  if constexpr (V == 8) {
    const float4 a = reinterpret_cast<const float4*>(plane)[vec], b = reinterpret_cast<const float4*>(plane)[nvec + vec];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    f[0] = plane[vec];
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
// t + 2T, ... (T threads, N vectors of V elements at most).  A team goes
// through consecutive rows, or through every teams-th row of its block's
// share, and asks for its next row as soon as it has taken the present one
// out of the load registers, before that row's sums.
//
// SHARED: the block folds the factors of a modulation group into shared memory
// and its teams read them from there; else every thread keeps those of its own
// channels in registers and folds them anew where the group changes.
template <typename TX, typename TY, int V, int N, bool RES, bool SHARED>
__global__ void __launch_bounds__(kNormThreads, 1) norm_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) float factors[];
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

  // this block's rows (SHARED) or this team's
  const long long parts = SHARED ? gridDim.x : static_cast<long long>(gridDim.x) * teams;
  const long long part = SHARED ? blockIdx.x : static_cast<long long>(blockIdx.x) * teams + team.index;
  const long long begin = rows * part / parts, end = rows * (part + 1) / parts;

  float A[SHARED ? 1 : N][V], Bv[SHARED ? 1 : N][V];        // of pre
  float PA[SHARED || !RES ? 1 : N][V], PB[SHARED || !RES ? 1 : N][V];   // of post and gate
  Raw<TX, V> rx[N];
  Raw<TY, V> ry[RES ? N : 1];
  auto load = [&](long long row) {
    const int b = static_cast<int>(row / p.L);
    const int l = static_cast<int>(row - static_cast<long long>(b) * p.L);
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
  };

  auto do_row = [&](long long row, int b, int l, long long next) {
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
        float x[V], a[V], c[V];
        if (!on[i]) {
#pragma unroll
          for (int j = 0; j < V; ++j) v[i][j] = 0.f;
          continue;
        }
        widen(rx[i], x);
        if constexpr (SHARED) {
          get_factor<V>(factors + 2 * p.C, nvec, tid + i * T, a);
          if (p.post_bias.p) get_factor<V>(factors + 3 * p.C, nvec, tid + i * T, c);
          else
#pragma unroll
            for (int j = 0; j < V; ++j) c[j] = 0.f;
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) a[j] = PA[i][j], c[j] = PB[i][j];
        }
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] = fmaf(p.rs, x[j], fmaf(v[i][j], a[j], c[j]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (on[i]) widen(rx[i], v[i]);
        else
#pragma unroll
          for (int j = 0; j < V; ++j) v[i][j] = 0.f;
      }
    }
    if (next < end) load(next);
    if constexpr (RES) {
      if (p.xo) {
        TX* op = static_cast<TX*>(p.xo) + b * p.xo_sb + l * p.xo_sl;
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (on[i]) store_row(op + (tid + i * T) * V, v[i]);
      }
      if (!p.h && !p.q) return;
    }
    normalise<V, N>(team, p.pre, p.pre_eps, p.C, on, v);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!on[i]) continue;
      float a[V], c[V];
      if constexpr (SHARED) {
        get_factor<V>(factors, nvec, tid + i * T, a);
        get_factor<V>(factors + p.C, nvec, tid + i * T, c);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) a[j] = A[i][j], c[j] = Bv[i][j];
      }
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = fmaf(v[i][j], a[j], c[j]);
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
  };

  if constexpr (SHARED) {
    long long have = -1;   // the row in the load registers
    for (long long s0 = begin; s0 < end;) {
      const int b = static_cast<int>(s0 / p.L);
      const int l = static_cast<int>(s0 - static_cast<long long>(b) * p.L);
      const long long s1 = min(end, s0 + (p.group - l % p.group));   // the group's end
      if (s0 + team.index < s1 && have != s0 + team.index) load(have = s0 + team.index);
      __syncthreads();   // the factors of the group before have been read
      for (int vec = threadIdx.x; vec < nvec; vec += blockDim.x) {
        float a[1][V], c[1][V];
        fold_pre<V, 1>(p, b, l, vec * V, 0, a, c);
        put_factor<V>(factors, nvec, vec, a[0]);
        put_factor<V>(factors + p.C, nvec, vec, c[0]);
        if constexpr (RES) {
          fold_post<V, 1>(p, b, l, vec * V, 0, a, c);
          put_factor<V>(factors + 2 * p.C, nvec, vec, a[0]);
          if (p.post_bias.p) put_factor<V>(factors + 3 * p.C, nvec, vec, c[0]);
        }
      }
      __syncthreads();
      for (long long row = s0 + team.index; row < s1; row += teams) {
        if (have != row) load(row);
        have = row + teams < s1 ? row + teams : s1 + team.index;
        do_row(row, b, l + static_cast<int>(row - s0), have);
      }
      s0 = s1;
    }
  } else {
    if (begin < end) load(begin);
    int until = 0, of = -1;   // the factors hold for the tokens below `until` of batch element `of`
    for (long long row = begin; row < end; ++row) {
      const int b = static_cast<int>(row / p.L);
      const int l = static_cast<int>(row - static_cast<long long>(b) * p.L);
      if (b != of || l >= until) {
        fold_pre<V, N>(p, b, l, tid * V, T * V, A, Bv);
        if constexpr (RES) fold_post<V, N>(p, b, l, tid * V, T * V, PA, PB);
        of = b;
        until = l - l % p.group + p.group;
      }
      do_row(row, b, l, row + 1);
    }
  }
}

}  // namespace solattn
