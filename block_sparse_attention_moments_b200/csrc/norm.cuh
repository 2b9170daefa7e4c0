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
//   s = max|h| / 127,  q = 127 h / max|h| to the nearest whole number, ties to even
//
// Everything between the loads and the stores is fp32 in registers: the row is
// read once, the variance is the mean square of the centred values (no
// difference of large sums), and h comes from the x' before its rounding.
// The parts that multiply and add along the channels are folded:
//   h = n * A + B   with A = weight * (1 + scale),  B = bias * (1 + scale) + shift
//   x' = rs * x + n_y * PA + PB  with PA = gate * post_weight, PB = gate * post_bias
//
// Bound by memory where there are many rows.  75600 rows of 5120, share of the
// copy rate (6.56 TB/s): bf16 norm 266 us (89%), fp32 residual and bf16 output
// with the next norm 738 us (96%), the same all in bf16 490 us (96%), fp32 to 8
// bits 335 us (88%; a rounding that misses ties took 316), the attention's
// head-major output to 8 bits 216 us (82%).
// 10166 rows of 1544 with a group of 391 each take 17.6 us (54%): a launch, the
// folding of two groups and five turns of each team.  Rows of odd width go
// element by element: 2062 of 1285 15.7 us (21%).
#pragma once

#include "rows.cuh"
#include "sm100_ptx.cuh"

namespace solattn {

constexpr int kNormRingThreads = 512;

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
  int inner_shift;                // log2 of x_inner, where the ring kernel reads pieces
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
__device__ __forceinline__ void put_factor(float* plane, int nvec, int vec, const float (&f)[8]) {
  reinterpret_cast<float4*>(plane)[vec] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(plane)[nvec + vec] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void get_factor(const float* plane, int nvec, int vec, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(plane)[vec], b = reinterpret_cast<const float4*>(plane)[nvec + vec];
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// Normalises R rows that the team holds in registers (no weight or bias).
template <int R, int V, int N, class Team>
__device__ __forceinline__ void normalise(Team& t, int kind, float eps, const NormParams& p, const bool (&on)[N],
                                          float (&v)[R][N][V]) {
  if (kind == kNormNone) return;
  float x[R];
  if (kind == kNormLayer) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < N; ++i) sum_v<V>(s, v[r][i]);   // zero outside the row
      x[r] = s.x + s.y;
    }
    t.template sum<R>(x);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float mean = divide_by(x[r], p.channels, p.inv_channels);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (on[i]) add_s<V>(v[r][i], -mean);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) sum_sq<V>(s, v[r][i]);
    x[r] = s.x + s.y;
  }
  t.template sum<R>(x);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float f = rsqrtf(fmaf(x[r], p.inv_channels, eps));
#pragma unroll
    for (int i = 0; i < N; ++i) mul_s<V>(v[r][i], f);
  }
}

template <int V, int N, bool WIDE, typename T>
__device__ __forceinline__ void store_vectors(T* p, const bool (&on)[N], const float (&v)[N][V]) {
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      uint4 u[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        u[h] = make_uint4(narrow2<T>(v[i + h][0], v[i + h][1]), narrow2<T>(v[i + h][2], v[i + h][3]),
                          narrow2<T>(v[i + h][4], v[i + h][5]), narrow2<T>(v[i + h][6], v[i + h][7]));
      st_row_v8(p + i * 32 * V, u[0], u[1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (on[i]) store_row(p + i * 32 * V, v[i]);
  }
}

// What happens to R rows v = x' (unrounded) of a team, tokens l, l + 1 of batch
// element b, of which those with `keep` are its: x' is written, normed,
// modulated with the factors that pre(i, a, c) gives, and written as h and in
// 8 bits.
// A thread's vectors are first, first + 32, ...; WIDE: pairs of neighbours,
// first, first + 1, first + 64, first + 65, ..., stored as one.
template <typename TX, typename TY, int R, int V, int N, bool RES, bool WIDE, class Team, class Pre>
__device__ __forceinline__ void emit_rows(const NormParams& p, Team& team, unsigned row, int b, int l, int first,
                                          const bool (&keep)[R], const bool (&on)[N], float (&v)[R][N][V], Pre pre) {
  if constexpr (RES) {
    if (p.xo) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (!keep[r]) continue;
        TX* op = static_cast<TX*>(p.xo) + b * p.xo_sb + (l + r) * p.xo_sl + first * V;
        store_vectors<V, N, WIDE>(op, on, v[r]);
      }
    }
    if (!p.h && !p.q) return;
  }
  normalise<R, V, N>(team, p.pre, p.pre_eps, p, on, v);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!on[i]) continue;
    float a[V], c[V];
    pre(i, a, c);
#pragma unroll
    for (int r = 0; r < R; ++r) fma_v<V>(v[r][i], v[r][i], a, c);
  }
  if (p.h) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (!keep[r]) continue;
      TY* hp = static_cast<TY*>(p.h) + b * p.h_sb + (l + r) * p.h_sl + first * V;
      store_vectors<V, N, WIDE>(hp, on, v[r]);
    }
  }
  if (p.q) {
    float amax[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (!on[i]) continue;
#pragma unroll
        for (int j = 0; j < V; j += 2) m = max_abs3(m, v[r][i][j], V > 1 ? v[r][i][j + V / 8] : 0.f);
      }
      amax[r] = m;
    }
    team.template max<R>(amax);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (!keep[r]) continue;
      // A row of zeros has the scale 0 and zeros; one with an infinity or a NaN
      // a scale that is not finite, and zeros too.  A row whose largest value is
      // below 2^-100 or above 2^100 is multiplied by a power of two first, so that
      // 127 / amax and its second term stay in range; what that rounds is far
      // below a half of a step.
      Up8 up{0.f, 0.f};
      if (amax[r] >= 0x1p-100f && amax[r] <= 0x1p100f) {
        up = up_s8(amax[r]);
      } else {
        const bool live = amax[r] > 0.f && amax[r] <= 3.402823466e38f;
        const float by = !live ? 0.f : amax[r] < 1.f ? 0x1p100f : 0x1p-100f;
        if (live) up = up_s8(amax[r] * by);
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j) v[r][i][j] = live ? v[r][i][j] * by : 0.f;
      }
      int8_t* qp = p.q + (row + r) * p.q_sl + first * V;
      if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const uint2 a = pack_s8(v[r][i], up), c = pack_s8(v[r][i + 1], up);
          *reinterpret_cast<uint4*>(qp + i * 32 * V) = make_uint4(a.x, a.y, c.x, c.y);
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (on[i]) store_s8<V>(qp + i * 32 * V, v[r][i], up);
      }
      if (first == 0) p.q_scale[row + r] = amax[r] / 127.f;
    }
  }
}

// Few rows, short groups, rows that vectors cannot read.  One team to a row;
// each warp has 32 N consecutive vectors of V elements, each thread N of them
// and, in registers, the folded factors of its channels, which it folds anew
// where the group changes.  A team goes through consecutive rows and asks for
// the next one as soon as it has taken the present one out of the load
// registers, before its sums.  Bound by the latency of a row's loads and sums;
// two blocks to an SM hide some of it (2062 rows of 1285 channels: 21.4 us with
// one, 15.8 with two).
template <typename TX, typename TY, int V, int N, bool RES, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS <= 352 ? 2 : 1) norm_kernel(const __grid_constant__ NormParams p) {
  using Team1 = Team<THREADS / 32, 1>;
  __shared__ __align__(16) float slots[Team1::shared(128, 0)];   // more than one team: 128 threads
  Team1 team;
  team.make(p.warps, slots, Team1::shared(128, 0));
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
    float v[1][N][V];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (on[i]) {
        if constexpr (RES) widen(ry[i], v[0][i]);
        else widen(rx[i], v[0][i]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[0][i][j] = 0.f;
      }
    }
    if constexpr (RES) {
      normalise<1, V, N>(team, p.post, p.post_eps, p, on, v);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (!on[i]) continue;
        float x[V];
        widen(rx[i], x);
        fma_v<V>(v[0][i], v[0][i], PA[i], PB[i]);
        fma_s<V>(v[0][i], x, p.rs, v[0][i]);
      }
    }
    if (row + 1 < end) load(row + 1);
    const bool keep[1] = {true};
    emit_rows<TX, TY, 1, V, N, RES, false>(p, team, row, b, l, first, keep, on, v, [&](int i, float(&a)[V], float(&c)[V]) {
#pragma unroll
      for (int j = 0; j < V; ++j) a[j] = A[i][j], c[j] = Bv[i][j];
    });
  }
}

// Many rows of long groups.  The block folds the factors of a group into
// shared memory and its teams, each with every teams-th R rows of the block's
// share, read them from there, once for R rows.
// R = 1: a thread's vectors are 32 bytes (8 of fp32, or two neighbours of 8 of
// a 16-bit type: WIDE), and the next row is on its way in registers.  R = 2,
// for 16-bit rows that 32-byte vectors do not fill: 16 bytes a vector, and the
// rows come through a ring of p.depth stages of R rows in shared memory by
// asynchronous copies, each warp's part by that warp.  75600 x 5120:
//   fp32 to 8 bits           R = 1 335 us; before ties were held 316, ring 454
//   fp32 with bf16 output    R = 1 737 us, ring 830
//   bf16                     R = 1 266 us with 32-byte vectors, 362 with 16, ring 287
// FULL: the teams' threads have exactly the row's vectors.  R rows that a
// group's end divides are taken twice, once with each group's factors, and
// each of them is kept once.
template <typename TX, typename TY, int R, int N, bool RES, bool FULL, int WARPS>
__global__ void __launch_bounds__(kNormRingThreads, 1) norm_ring_kernel(const __grid_constant__ NormParams p) {
  constexpr int V = 8;
  constexpr int kX = N * 32 * V * sizeof(TX), kY = RES ? N * 32 * V * sizeof(TY) : 0;   // bytes of a warp's row
  constexpr bool WIDE = R == 1 && sizeof(TX) == 2;
  static_assert(!WIDE || FULL, "pairs of vectors fill the row");
  constexpr bool RING = R > 1;
  constexpr int kStage = R * (kX + kY);
  using TeamR = Team<WARPS, R>;
  constexpr int kTeamSlots = TeamR::shared(kNormRingThreads, 1);
  extern __shared__ __align__(16) float factors[];
  __shared__ __align__(16) float slots[kTeamSlots];
  TeamR team;
  team.make(p.warps, slots, kTeamSlots);
  const int lane = threadIdx.x % 32;
  const int teams = blockDim.x / 32 / team.warps;
  const int first = team.warp * 32 * N + (WIDE ? 2 : 1) * lane;
  const int nvec = p.C / V;
  // where a vector's factors lie (WIDE: even vectors, then odd ones, as lanes read every other one)
  auto place = [&](int vec) { return WIDE ? (vec >> 1) + (vec & 1 ? nvec >> 1 : 0) : vec; };
  const int mine = WIDE ? (team.warp * 32 * N >> 1) + lane : first;
  auto factor = [&](int i) { return WIDE ? mine + (i >> 1) * 32 + (i & 1 ? nvec >> 1 : 0) : mine + i * 32; };
  const unsigned L = p.L, rows = p.B * L;   // below 2^31
  const int planes = RES ? (p.post_bias.p ? 4 : 3) : 2;
  uint8_t* ring = reinterpret_cast<uint8_t*>(factors + planes * p.C) + (threadIdx.x / 32) * p.depth * kStage;

  bool on[N];
#pragma unroll
  for (int i = 0; i < N; ++i) on[i] = FULL || first + i * 32 < nvec;

  const unsigned begin = static_cast<unsigned long long>(rows) * blockIdx.x / gridDim.x;
  const unsigned end = static_cast<unsigned long long>(rows) * (blockIdx.x + 1) / gridDim.x;

  // the first of the rows that are to be fetched next
  unsigned next = begin + R * team.index;
  int nb = next / L, nl = next - nb * L;
  auto advance = [&]() {
    next += R * teams;
    nl += R * teams;
    while (nl >= p.L && next < end) nl -= p.L, ++nb;
  };
  Raw<TX, V> rx[RING ? 1 : N];          // without a ring: the row on its way
  Raw<TY, V> ry[RING || !RES ? 1 : N];
  auto load = [&](int stage) {
    if constexpr (!RING) {
      if (next < end) {
        const TX* xp = static_cast<const TX*>(p.x) + nb * p.x_sb + nl * p.x_sl;
        const TY* yp = static_cast<const TY*>(p.y) + nb * p.y_sb + nl * p.y_sl + first * V;
        auto piece = [&](int c) {   // channel c of a row of pieces
          return xp + (c >> p.inner_shift) * p.x_sh + (c & ((1 << p.inner_shift) - 1));
        };
        if constexpr (WIDE) {
#pragma unroll
          for (int i = 0; i < N; i += 2) {
            const int c = (first + i * 32) * V;
            ld_row_v8(p.x_inner == p.C ? xp + c : piece(c), rx[i].r[0], rx[i + 1].r[0]);
            if constexpr (RES) ld_row_v8(yp + i * 32 * V, ry[i].r[0], ry[i + 1].r[0]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            if (!on[i]) continue;
            const int c = (first + i * 32) * V;
            load_raw(rx[i], p.x_inner == p.C ? xp + c : piece(c));
            if constexpr (RES) load_raw(ry[i], yp + i * 32 * V);
          }
        }
      }
      advance();
      return cp_async_commit();
    }
    constexpr int kPieceX = 16 / sizeof(TX), kPieceY = 16 / sizeof(TY);   // channels of a 16-byte piece
    const int c0 = team.warp * 32 * N * V;                                // the warp's first channel
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (next + r >= end) continue;
      const bool wrap = nl + r >= p.L;   // the row after a batch element's last (R <= 2)
      const long long b = nb + wrap, l = wrap ? 0 : nl + r;
      const uint32_t dst = smem_u32(ring + stage * kStage + r * (kX + kY)) + lane * 16;
      const TX* xp = static_cast<const TX*>(p.x) + b * p.x_sb + l * p.x_sl;
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
              cp_async_16(dst + i * 32 * V * sizeof(TX) + 512 * h,
                          xp + (c >> p.inner_shift) * p.x_sh + (c & ((1 << p.inner_shift) - 1)));
          }
      }
      if constexpr (RES) {
        const TY* yl = static_cast<const TY*>(p.y) + b * p.y_sb + l * p.y_sl + c0 + lane * kPieceY;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int h = 0; h < V / kPieceY; ++h)
            if (FULL || c0 + i * 32 * V + (lane + 32 * h) * kPieceY < p.C)
              cp_async_16(dst + kX + i * 32 * V * sizeof(TY) + 512 * h, yl + i * 32 * V + 32 * h * kPieceY);
      }
    }
    advance();
    cp_async_commit();   // also where there is nothing to copy: groups are counted
  };

  unsigned row = begin + R * team.index;
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
      put_factor(factors, nvec, place(vec), a[0]);
      put_factor(factors + p.C, nvec, place(vec), c[0]);
      if constexpr (RES) {
        fold_post<V, 1>(p, b, l0, vec * V, 0, a, c);
        put_factor(factors + 2 * p.C, nvec, place(vec), a[0]);
        if (p.post_bias.p) put_factor(factors + 3 * p.C, nvec, place(vec), c[0]);
      }
    }
    __syncthreads();
    while (row < s1) {
      // All but the depth - 1 youngest groups are complete: these rows have come.
      // (Rows in registers keep the empty groups and the warp's meetings: without
      // them the compiler's order of the loads costs 7%.)
      if (p.depth == 1) cp_async_wait<0>();
      else if (p.depth == 2) cp_async_wait<1>();
      else if (p.depth == 3) cp_async_wait<2>();
      else cp_async_wait<3>();
      // A team that begins a row together reads and writes in longer runs: with
      // a block's output, 75600 x 5120 bf16 533 us without this meeting and 490
      // with it, fp32 without a norm 636 and 607; an fp32 stream with a norm
      // behind it (739 without, 791 with) and lone norms (270, 280) do without.
      if (RES && (WIDE || (!p.h && !p.q))) team.sync();
      else __syncwarp();
      [[maybe_unused]] const uint8_t* src = ring + stage * kStage;
      bool keep[R];
#pragma unroll
      for (int r = 0; r < R; ++r) keep[r] = R == 1 || (row + r >= s0 && row + r < s1);
      float v[R][N][V];
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (on[i]) {
            if constexpr (!RING && RES) widen(ry[i], v[r][i]);
            else if constexpr (!RING) widen(rx[i], v[r][i]);
            else if constexpr (RES) take_staged<TY>(src + r * (kX + kY) + kX, i * 32 + lane, v[r][i]);
            else take_staged<TX>(src + r * (kX + kY), i * 32 + lane, v[r][i]);
          } else {
#pragma unroll
            for (int j = 0; j < V; ++j) v[r][i][j] = 0.f;
          }
        }
      }
      if constexpr (RES) {
        normalise<R, V, N>(team, p.post, p.post_eps, p, on, v);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (!on[i]) continue;
          float a[V], c[V];
          get_factor(factors + 2 * p.C, nvec, factor(i), a);
          if (p.post_bias.p) get_factor(factors + 3 * p.C, nvec, factor(i), c);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float x[V];
            if (p.post_bias.p) fma_v<V>(v[r][i], v[r][i], a, c);
            else mul_v<V>(v[r][i], a);
            if constexpr (RING) take_staged<TX>(src + r * (kX + kY), i * 32 + lane, x);
            else widen(rx[i], x);
            fma_s<V>(v[r][i], x, p.rs, v[r][i]);
          }
        }
      }
      const bool again = R > 1 && row + R > s1 && s1 < end;   // some of these rows are the next group's
      const unsigned this_row = row;
      if (!again) {
        __syncwarp();   // all lanes have read the stage
        load(stage);
        stage = stage + 1 == p.depth ? 0 : stage + 1;
        row += R * teams;
      }
      emit_rows<TX, TY, R, V, N, RES, WIDE>(p, team, this_row, b, l0 + static_cast<int>(this_row - s0), first, keep, on, v,
                                      [&](int i, float(&a)[V], float(&c)[V]) {
                                        get_factor(factors, nvec, factor(i), a);
                                        get_factor(factors + p.C, nvec, factor(i), c);
                                      });
      if (again) break;
    }
    s0 = s1;
  }
  cp_async_wait<0>();
}

}  // namespace solattn
