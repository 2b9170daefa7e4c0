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
#include "sm100_ptx.cuh"

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
  int depth;                      // stages of the ring
  float channels, inv_channels;   // C and 1 / C
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
__device__ __forceinline__ void normalise(Team& t, int kind, float eps, const NormParams& p, const bool (&on)[N], float (&v)[N][V]) {
  if (kind == kNormNone) return;
  if (kind == kNormLayer) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) sum_v<V>(s, v[i]);   // zero outside the row
    const float mean = divide_by(team_sum(t, s.x + s.y), p.channels, p.inv_channels);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (on[i]) add_s<V>(v[i], -mean);
  }
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < N; ++i) sum_sq<V>(s, v[i]);
  const float r = rsqrtf(fmaf(team_sum(t, s.x + s.y), p.inv_channels, eps));
#pragma unroll
  for (int i = 0; i < N; ++i) mul_s<V>(v[i], r);
}

// What happens to a row v = x' (unrounded) of a team: x' is written, normed,
// modulated with the factors that pre(i, a, c) gives, and written as h and in
// 8 bits.
template <typename TX, typename TY, int V, int N, bool RES, class Pre>
__device__ __forceinline__ void emit_row(const NormParams& p, Team& team, unsigned row, int b, int l, int first,
                                         const bool (&on)[N], float (&v)[N][V], Pre pre) {
  if constexpr (RES) {
    if (p.xo) {
      TX* op = static_cast<TX*>(p.xo) + b * p.xo_sb + l * p.xo_sl;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (on[i]) store_row(op + (first + i * 32) * V, v[i]);
    }
    if (!p.h && !p.q) return;
  }
  normalise<V, N>(team, p.pre, p.pre_eps, p, on, v);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!on[i]) continue;
    float a[V], c[V];
    pre(i, a, c);
    fma_v<V>(v[i], v[i], a, c);
  }
  if (p.h) {
    TY* hp = static_cast<TY*>(p.h) + b * p.h_sb + l * p.h_sl;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (on[i]) store_row(hp + (first + i * 32) * V, v[i]);
  }
  if (p.q) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (on[i]) m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
    const float amax = __uint_as_float(team_max(team, m));
    // q = h * (127 / amax).  A row of zeros has the scale 0; of one with an
    // infinity or a NaN the scale is not finite.  Both get the factor 0, and
    // what is NaN then becomes 0 as a whole number.  Below 2^-120 the row is
    // scaled up first, as 127 / amax would overflow.
    const bool tiny = amax < 0x1p-120f;
    if (tiny) {
#pragma unroll
      for (int i = 0; i < N; ++i) mul_s<V>(v[i], 0x1p100f);
    }
    const float up = amax > 0.f && amax <= 3.402823466e38f ? 127.f / (tiny ? amax * 0x1p100f : amax) : 0.f;
    int8_t* qp = p.q + row * p.q_sl;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!on[i]) continue;
      mul_s<V>(v[i], up);
      if constexpr (V == 8) {
        int k[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) k[j] = __float2int_rn(v[i][j]);
        *reinterpret_cast<uint2*>(qp + (first + i * 32) * 8) =
            make_uint2(pack_s8(k[0], k[1], k[2], k[3]), pack_s8(k[4], k[5], k[6], k[7]));
      } else {
        qp[first + i * 32] = static_cast<int8_t>(__float2int_rn(v[i][0]));
      }
    }
    if (first == 0) p.q_scale[row] = amax / 127.f;
  }
}

// Few rows, short groups, rows that vectors cannot read.  One team to a row;
// each warp has 32 N consecutive vectors of V elements, each thread N of them
// and, in registers, the folded factors of its channels, which it folds anew
// where the group changes.  A
// team goes through consecutive rows and asks for the next one as soon as it
// has taken the present one out of the load registers, before its sums.
template <typename TX, typename TY, int V, int N, bool RES, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ __align__(16) float slots[team_slots(THREADS, 1)];
  Team team;
  make_team<1>(team, p.warps, slots, team_slots(THREADS, 1));
  const int teams = blockDim.x / 32 / p.warps;
  const int first = team.warp * 32 * N + threadIdx.x % 32;   // this thread's vectors: first, first + 32, ...
  const int nvec = p.C / V;
  const unsigned L = p.L, rows = p.B * L;   // below 2^31

  bool on[N];
#pragma unroll
  for (int i = 0; i < N; ++i) on[i] = first + i * 32 < nvec;

  const unsigned long long parts = gridDim.x * teams, part = blockIdx.x * teams + team.index;
  const unsigned begin = rows * part / parts, end = rows * (part + 1) / parts;

  float A[N][V], Bv[N][V];                            // of pre
  float PA[RES ? N : 1][V], PB[RES ? N : 1][V];       // of post and gate
  Raw<TX, V> rx[N];
  Raw<TY, V> ry[RES ? N : 1];
  auto load = [&](unsigned row) {
    const int b = row / L;
    const int l = row - b * L;
    const TX* xp = static_cast<const TX*>(p.x) + b * p.x_sb + l * p.x_sl;
    if (p.x_inner == p.C) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (on[i]) load_raw(rx[i], xp + (first + i * 32) * V);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (first + i * 32) * V;
        if (on[i]) load_raw(rx[i], xp + (c / p.x_inner) * p.x_sh + c % p.x_inner);
      }
    }
    if constexpr (RES) {
      const TY* yp = static_cast<const TY*>(p.y) + b * p.y_sb + l * p.y_sl;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (on[i]) load_raw(ry[i], yp + (first + i * 32) * V);
    }
  };

  if (begin < end) load(begin);
  __syncthreads();   // the team's slots are clear
  int until = 0, of = -1;   // the factors hold for the tokens below `until` of batch element `of`
  for (unsigned row = begin; row < end; ++row) {
    const int b = row / L;
    const int l = row - b * L;
    if (b != of || l >= until) {
      fold_pre<V, N>(p, b, l, first * V, 32 * V, A, Bv);
      if constexpr (RES) fold_post<V, N>(p, b, l, first * V, 32 * V, PA, PB);
      of = b;
      until = l - l % p.group + p.group;
    }
    float v[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (on[i]) {
        if constexpr (RES) widen(ry[i], v[i]);
        else widen(rx[i], v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] = 0.f;
      }
    }
    if constexpr (RES) {
      normalise<V, N>(team, p.post, p.post_eps, p, on, v);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (!on[i]) continue;
        float x[V];
        widen(rx[i], x);
        fma_v<V>(v[i], v[i], PA[i], PB[i]);
        fma_s<V>(v[i], x, p.rs, v[i]);
      }
    }
    if (row + 1 < end) load(row + 1);
    emit_row<TX, TY, V, N, RES>(p, team, row, b, l, first, on, v, [&](int i, float(&a)[V], float(&c)[V]) {
#pragma unroll
      for (int j = 0; j < V; ++j) a[j] = A[i][j], c[j] = Bv[i][j];
    });
  }
}

// Many rows of long groups.  The block folds the factors of a group into
// shared memory and its teams, each with every teams-th row of the block's
// share, read them from there.  Rows come through a ring of p.depth stages in
// shared memory by asynchronous copies, each warp's part by that warp: rows on
// their way cost no registers, and no barrier but the warp's own.
template <typename TX, typename TY, int N, bool RES, bool FULL, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) norm_ring_kernel(const __grid_constant__ NormParams p) {
  constexpr int V = 8;
  constexpr int kX = N * 32 * V * sizeof(TX), kY = RES ? N * 32 * V * sizeof(TY) : 0;   // bytes of a warp's stage
  extern __shared__ __align__(16) float factors[];
  __shared__ __align__(16) float slots[team_slots(THREADS, 1)];
  Team team;
  make_team<1>(team, p.warps, slots, team_slots(THREADS, 1));
  const int lane = threadIdx.x % 32;
  const int teams = blockDim.x / 32 / p.warps;
  const int first = team.warp * 32 * N + threadIdx.x % 32;   // this thread's vectors: first, first + 32, ...
  const int nvec = p.C / V;
  const unsigned L = p.L, rows = p.B * L;   // below 2^31
  const int planes = RES ? (p.post_bias.p ? 4 : 3) : 2;
  uint8_t* ring = reinterpret_cast<uint8_t*>(factors + planes * p.C) + (threadIdx.x / 32) * p.depth * (kX + kY);

  bool on[N];
#pragma unroll
  for (int i = 0; i < N; ++i) on[i] = first + i * 32 < nvec;

  const unsigned begin = static_cast<unsigned long long>(rows) * blockIdx.x / gridDim.x;
  const unsigned end = static_cast<unsigned long long>(rows) * (blockIdx.x + 1) / gridDim.x;

  constexpr int kPieceX = 16 / sizeof(TX), kPieceY = 16 / sizeof(TY);   // channels of a 16-byte piece
  const int c0 = team.warp * 32 * N * V;                                // the warp's first channel
  // the row that the next copies bring: batch element, token, and whether it is the block's
  unsigned next = begin + team.index;
  int nb = next / L, nl = next - nb * L;
  auto load = [&](int stage) {
    if (next < end) {
      const uint32_t dst = smem_u32(ring + stage * (kX + kY)) + lane * 16;
      const TX* xp = static_cast<const TX*>(p.x) + nb * p.x_sb + nl * p.x_sl;
      if (p.x_inner == p.C) {
        const TX* xl = xp + c0 + lane * kPieceX;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int h = 0; h < V / kPieceX; ++h)
            if (FULL || c0 + i * 32 * V + (lane + 32 * h) * kPieceX < p.C)
              cp_async_16(dst + i * 32 * V * sizeof(TX) + 512 * h, xl + i * 32 * V + 32 * h * kPieceX);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int h = 0; h < V / kPieceX; ++h) {
            const int c = c0 + i * 32 * V + (lane + 32 * h) * kPieceX;
            if (FULL || c < p.C)
              cp_async_16(dst + i * 32 * V * sizeof(TX) + 512 * h, xp + (c / p.x_inner) * p.x_sh + c % p.x_inner);
          }
      }
      if constexpr (RES) {
        const TY* yl = static_cast<const TY*>(p.y) + nb * p.y_sb + nl * p.y_sl + c0 + lane * kPieceY;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int h = 0; h < V / kPieceY; ++h)
            if (FULL || c0 + i * 32 * V + (lane + 32 * h) * kPieceY < p.C)
              cp_async_16(dst + kX + i * 32 * V * sizeof(TY) + 512 * h, yl + i * 32 * V + 32 * h * kPieceY);
      }
      next += teams;
      nl += teams;
      while (nl >= p.L) nl -= p.L, ++nb;
    }
    cp_async_commit();   // also where there is nothing to copy: groups are counted
  };

  unsigned row = begin + team.index;
  for (int s = 0; s < p.depth; ++s) load(s);
  int stage = 0;
  for (unsigned s0 = begin; s0 < end;) {
    const int b = s0 / L;
    const int l0 = s0 - b * L;
    const unsigned s1 = min(end, s0 + (p.group - l0 % p.group));   // the group's end
    __syncthreads();   // the factors of the group before have been read
    for (int vec = threadIdx.x; vec < nvec; vec += blockDim.x) {
      float a[1][V], c[1][V];
      fold_pre<V, 1>(p, b, l0, vec * V, 0, a, c);
      put_factor<V>(factors, nvec, vec, a[0]);
      put_factor<V>(factors + p.C, nvec, vec, c[0]);
      if constexpr (RES) {
        fold_post<V, 1>(p, b, l0, vec * V, 0, a, c);
        put_factor<V>(factors + 2 * p.C, nvec, vec, a[0]);
        if (p.post_bias.p) put_factor<V>(factors + 3 * p.C, nvec, vec, c[0]);
      }
    }
    __syncthreads();
    for (; row < s1; row += teams) {
      // all but the depth - 1 youngest groups are complete: this row has come
      if (p.depth == 1) cp_async_wait<0>();
      else if (p.depth == 2) cp_async_wait<1>();
      else if (p.depth == 3) cp_async_wait<2>();
      else cp_async_wait<3>();
      __syncwarp();
      const uint8_t* src = ring + stage * (kX + kY);
      float v[N][V];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (on[i]) {
          if constexpr (RES) take_staged<TY>(src + kX, i * 32 + lane, v[i]);
          else take_staged<TX>(src, i * 32 + lane, v[i]);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) v[i][j] = 0.f;
        }
      }
      if constexpr (RES) {
        normalise<V, N>(team, p.post, p.post_eps, p, on, v);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (!on[i]) continue;
          float x[V], a[V];
          get_factor<V>(factors + 2 * p.C, nvec, first + i * 32, a);
          if (p.post_bias.p) {
            float c[V];
            get_factor<V>(factors + 3 * p.C, nvec, first + i * 32, c);
            fma_v<V>(v[i], v[i], a, c);
          } else {
            mul_v<V>(v[i], a);
          }
          take_staged<TX>(src, i * 32 + lane, x);
          fma_s<V>(v[i], x, p.rs, v[i]);
        }
      }
      __syncwarp();   // all lanes have read the stage
      load(stage);
      stage = stage + 1 == p.depth ? 0 : stage + 1;
      emit_row<TX, TY, V, N, RES>(p, team, row, b, l0 + (row - s0), first, on, v,
                                  [&](int i, float(&a)[V], float(&c)[V]) {
                                    get_factor<V>(factors, nvec, first + i * 32, a);
                                    get_factor<V>(factors + p.C, nvec, first + i * 32, c);
                                  });
    }
    s0 = s1;
  }
  cp_async_wait<0>();
}

}  // namespace solattn
