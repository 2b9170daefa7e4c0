// rope.cuh — queries, keys and values of one projection, made ready for the
// attention: RMS norm of q and k, rotary positions with several axes, and the
// head-major layout [B, H, L, d].
//
// A head's d channels form d / 2 pairs (a, b), and pair i turns by the angle
//   t = position[axis(i)] * freq(i),   (a, b) -> (a cos t - b sin t, a sin t + b cos t)
// with the pairs (2i, 2i + 1) ("interleaved") or (i, i + d / 2) ("half").  The
// position of a token has up to four axes: given for each token, or (frame,
// row, column) on a grid that the tokens fill in raster order; tokens behind
// the grid (text) do not turn.
//
// The angle is formed in fp64, in turns, and only its fraction is rounded to
// fp32: a position of 10^5 would cost an fp32 angle three of its digits.
#pragma once

#include <climits>

#include "rows.cuh"

namespace solattn {

enum : int { kRopeNormNone = 0, kRopeNormHead = 1, kRopeNormToken = 2 };
enum : int { kPosGrid = 0, kPosI32 = 1, kPosI64 = 2, kPosF32 = 3, kPosF64 = 4 };

constexpr int kRopeMaxD = 256;
constexpr int kRopeMaxAxes = 4;

struct RopeTensor {
  const void* in;       // [B, L, H, d], the channels of a head contiguous
  long long sb, sl, sh;
  void* out;            // contiguous [B, H, L, d]
  const void* weight;   // [d] or [H*d] (null: ones)
  int weight_dtype;
};

struct RopeParams {
  int B, L, H, d;
  RopeTensor q, k, v;   // v.in null: not wanted
  int norm;
  float eps;
  int half;             // pairing
  int pos_kind;
  const void* pos;      // [B, L, A]
  long long pos_sb, pos_sl, pos_sa;
  int grid_h, grid_w;
  long long grid_tokens, start;
  int warps;            // warps of a team
  double turns[kRopeMaxD / 2];        // frequency of a pair / (2 pi)
  unsigned char axis[kRopeMaxD / 2];  // axis of a pair
};

constexpr int kRopeThreads = 512;

__device__ __forceinline__ double rope_position(const RopeParams& p, int b, int l, int axis) {
  if (p.pos_kind == kPosGrid) {
    const long long i = p.start + l;
    if (i >= p.grid_tokens) return 0.0;
    const unsigned u = static_cast<unsigned>(i);   // a grid has fewer than 2^31 tokens
    const unsigned w = p.grid_w, hw = static_cast<unsigned>(p.grid_h) * w;
    return axis == 0 ? u / hw : axis == 1 ? (u % hw) / w : u % w;
  }
  const long long at = b * p.pos_sb + l * p.pos_sl + axis * p.pos_sa;
  if (p.pos_kind == kPosI32) return static_cast<const int*>(p.pos)[at];
  if (p.pos_kind == kPosI64) return static_cast<double>(static_cast<const long long*>(p.pos)[at]);
  if (p.pos_kind == kPosF32) return static_cast<const float*>(p.pos)[at];
  return static_cast<const double*>(p.pos)[at];
}

// A unit is 16 channels of a head, 8 pairs: two adjacent 16-byte vectors
// (interleaved) or two that lie d / 2 channels apart (half).
template <typename T>
struct RopeUnit {
  Raw<T, 8> a, b;
};

__device__ __forceinline__ void rope_rotate(bool half, const float (&cs)[8], const float (&sn)[8], float (&a)[8],
                                            float (&b)[8]) {
  if (half) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = a[j], y = b[j];
      a[j] = x * cs[j] - y * sn[j];
      b[j] = x * sn[j] + y * cs[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = a[2 * j], y = a[2 * j + 1];
      a[2 * j] = x * cs[j] - y * sn[j];
      a[2 * j + 1] = x * sn[j] + y * cs[j];
      const float u = b[2 * j], w = b[2 * j + 1];
      b[2 * j] = u * cs[4 + j] - w * sn[4 + j];
      b[2 * j + 1] = u * sn[4 + j] + w * cs[4 + j];
    }
  }
}

// One team to a token, all its heads.  Thread t of the team holds the units
// t, t + T, ... of q and of k (N at most); v is copied.
template <typename T, int N>
__global__ void __launch_bounds__(kRopeThreads, 1) rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ float smem[];
  __shared__ double turns[kRopeMaxD / 2];
  __shared__ float slots[2 * (kRopeThreads / 32)];
  Team team;
  team.warps = p.warps;
  team.index = (threadIdx.x / 32) / p.warps;
  team.warp = (threadIdx.x / 32) % p.warps;
  team.slots = slots + 2 * p.warps * team.index;
  team.turn = 0;
  const int teams = blockDim.x / 32 / p.warps;
  const int TT = p.warps * 32;
  const int tid = threadIdx.x - team.index * TT;
  const int d2 = p.d / 2;
  const int per_head = p.d / 16;
  const int units = p.H * per_head;
  // per team: cos and sin of the token's pairs, then (head norm) each unit's sums for q and k
  float* table = smem + team.index * (p.d + (p.norm == kRopeNormHead ? 2 * units : 0));
  float* sums = table + p.d;
  for (int i = threadIdx.x; i < d2; i += blockDim.x) turns[i] = p.turns[i];
  __syncthreads();

  const long long tokens = static_cast<long long>(p.B) * p.L;
  for (long long tok = static_cast<long long>(blockIdx.x) * teams + team.index; tok < tokens;
       tok += static_cast<long long>(gridDim.x) * teams) {
    const int b = static_cast<int>(tok / p.L);
    const int l = static_cast<int>(tok - static_cast<long long>(b) * p.L);
    RopeUnit<T> rq[N], rk[N];
    const T* qp = static_cast<const T*>(p.q.in) + b * p.q.sb + l * p.q.sl;
    const T* kp = static_cast<const T*>(p.k.in) + b * p.k.sb + l * p.k.sl;
    const int second = p.half ? d2 : 8;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = tid + i * TT;
      if (u >= units) continue;
      const int head = u / per_head, c = (u % per_head) * (p.half ? 8 : 16);
      load_raw(rq[i].a, qp + head * p.q.sh + c);
      load_raw(rq[i].b, qp + head * p.q.sh + c + second);
      load_raw(rk[i].a, kp + head * p.k.sh + c);
      load_raw(rk[i].b, kp + head * p.k.sh + c + second);
    }
    // the table of the previous token has been read by all of the team
    team_sync(team);
    for (int i = tid; i < d2; i += TT) {
      const double t = rope_position(p, b, l, p.axis[i]) * turns[i];
      float sn, cs;
      sincospif(2.f * static_cast<float>(t - rint(t)), &sn, &cs);
      table[i] = cs;
      table[d2 + i] = sn;
    }
    float mq = 1.f, mk = 1.f;   // with a token norm: 1 / rms
    if (p.norm != kRopeNormNone) {
      float sq = 0.f, sk = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int u = tid + i * TT;
        if (u >= units) continue;
        float a[8], c[8];
        float uq = 0.f, uk = 0.f;
        widen(rq[i].a, a);
        widen(rq[i].b, c);
#pragma unroll
        for (int j = 0; j < 8; ++j) uq = fmaf(a[j], a[j], fmaf(c[j], c[j], uq));
        widen(rk[i].a, a);
        widen(rk[i].b, c);
#pragma unroll
        for (int j = 0; j < 8; ++j) uk = fmaf(a[j], a[j], fmaf(c[j], c[j], uk));
        if (p.norm == kRopeNormHead) {
          sums[u] = uq;
          sums[units + u] = uk;
        }
        sq += uq;
        sk += uk;
      }
      if (p.norm == kRopeNormToken) {
        const float inv = 1.f / static_cast<float>(p.H * p.d);
        mq = rsqrtf(team_sum(team, sq) * inv + p.eps);
        mk = rsqrtf(team_sum(team, sk) * inv + p.eps);
      }
    }
    team_sync(team);   // the table (and the units' sums) are complete

    const long long head_stride = static_cast<long long>(p.L) * p.d;
    const long long out0 = (static_cast<long long>(b) * p.H * p.L + l) * p.d;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = tid + i * TT;
      if (u >= units) continue;
      const int head = u / per_head, c = (u % per_head) * (p.half ? 8 : 16);
      const int pair = (u % per_head) * 8;
      float cs[8], sn[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) cs[j] = table[pair + j], sn[j] = table[d2 + pair + j];
      if (p.norm == kRopeNormHead) {
        float sq = 0.f, sk = 0.f;
        for (int j = 0; j < per_head; ++j) {
          sq += sums[head * per_head + j];
          sk += sums[units + head * per_head + j];
        }
        const float inv = 1.f / static_cast<float>(p.d);
        mq = rsqrtf(sq * inv + p.eps);
        mk = rsqrtf(sk * inv + p.eps);
      }
      const long long o = out0 + head * head_stride + c;
      const int wc = p.norm == kRopeNormToken ? head * p.d + c : c;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const RopeTensor& x = which ? p.k : p.q;
        const float m = which ? mk : mq;
        float a[8], e[8], w[2][8];
        widen(which ? rk[i].a : rq[i].a, a);
        widen(which ? rk[i].b : rq[i].b, e);
        if (p.norm != kRopeNormNone) {
#pragma unroll
          for (int j = 0; j < 8; ++j) a[j] *= m, e[j] *= m;
          if (x.weight) {
            load_params<8, 2>(x.weight, x.weight_dtype, 0, wc, second, INT_MAX, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] *= w[0][j], e[j] *= w[1][j];
          }
        }
        rope_rotate(p.half, cs, sn, a, e);
        T* op = static_cast<T*>(x.out) + o;
        store_row(op, a);
        store_row(op + second, e);
      }
    }
    if (p.v.in) {
      const T* vp = static_cast<const T*>(p.v.in) + b * p.v.sb + l * p.v.sl;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int u = tid + i * TT;
        if (u >= units) continue;
        load_raw(rq[i].a, vp + (u / per_head) * p.v.sh + (u % per_head) * 16);
        load_raw(rq[i].b, vp + (u / per_head) * p.v.sh + (u % per_head) * 16 + 8);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int u = tid + i * TT;
        if (u >= units) continue;
        uint4* op = reinterpret_cast<uint4*>(static_cast<T*>(p.v.out) + out0 + (u / per_head) * head_stride +
                                             (u % per_head) * 16);
#pragma unroll
        for (int j = 0; j < Raw<T, 8>::kVecs; ++j) {
          op[j] = rq[i].a.r[j];
          op[Raw<T, 8>::kVecs + j] = rq[i].b.r[j];
        }
      }
    }
  }
}

}  // namespace solattn
