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
//
// Bound by memory: every value is read and written once.  75600 tokens of q, k
// and v of 40 heads of 128 in bf16, token norm: 4.64 GB in 755 to 770 us (6.0 to
// 6.15 TB/s; 708 us at the copy rate of 6.56); 4173 x 2 tokens of 16 heads of
// 64 with positions 24 us (15.6), where a team has two or three tokens and the
// first ones' latency is not hidden.  What brought it there from 1208 us: loads
// through shared memory instead of registers, tables and weights there without
// bank conflicts, one barrier a token, no division in the loop.
#pragma once

#include <climits>

#include "rows.cuh"
#include "sm100_ptx.cuh"

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
  int team_floats;      // shared memory of a team and parity
  int by_lanes;         // a head's items lie in lanes of one warp
  int packed;           // a token's heads lie one after the other in q, k and v
  int shared_weights;   // the weights are read from shared memory
  int staged;           // tensors that go through the stages: q, k and, where there is room, v
  int depth;            // stages of a team: 1 to 4
  float inv_channels;   // 1 / channels of a norm
  double turns[kRopeMaxD / 2];        // frequency of a pair / (2 pi)
  unsigned char axis[kRopeMaxD / 2];  // axis of a pair
};

constexpr int kRopeThreads = 768;

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

constexpr int kRopeVectors = 4;   // vectors of 8 channels that a thread holds of a tensor: 16 warps reach H*d = 16384

// Turns the pairs of two vectors whose channels pair up one by one (half), or
// those within one (interleaved).
__device__ __forceinline__ void rope_turn_half(float (&a)[8], float (&b)[8], const float (&cs)[8], const float (&sn)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = a[j], y = b[j];
    a[j] = x * cs[j] - y * sn[j];
    b[j] = x * sn[j] + y * cs[j];
  }
}
__device__ __forceinline__ void rope_turn(float (&a)[8], const float4& cs, const float4& sn) {
  const float c[4] = {cs.x, cs.y, cs.z, cs.w}, s[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float x = a[2 * j], y = a[2 * j + 1];
    a[2 * j] = x * c[j] - y * s[j];
    a[2 * j + 1] = x * s[j] + y * c[j];
  }
}

// One team to a token, all its heads.  An item is what turns together: a
// vector of 8 channels (interleaved) or two that lie d / 2 channels apart
// (half); each warp has 32 N consecutive items, each thread N of them.  Tokens
// come through p.depth stages in shared memory by asynchronous copies, each
// warp's part by that warp, and are read from there twice, for the norm and for
// the rotation.  The launch takes as many teams as fit and gives the stages what
// is left.  With v that is one stage up to 40 heads of 128: a team asks for its
// next token when it has read the present one, and the other teams' loads fill
// the time; without v it is two in most of the 16-bit cases.  The cosines and
// sines of a token are made by the team's first threads; their buffers alternate,
// so that the barrier of the norm's sum is the only one.
template <typename T, bool HALF, int WARPS>
__global__ void __launch_bounds__(kRopeThreads, 1) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int VECS = HALF ? 2 : 1, N = kRopeVectors / VECS;
  constexpr int kPieces = sizeof(T) / 2;                   // 16-byte pieces of a vector
  constexpr int kTensor = kRopeVectors * 32 * 8 * sizeof(T);   // bytes of a warp's part of a tensor
  extern __shared__ __align__(16) float smem[];
  __shared__ double turns[kRopeMaxD / 2];
  using Team2 = Team<WARPS, 2>;
  constexpr int kTeamSlots = Team2::shared(kRopeThreads, WARPS == 1 ? 0 : WARPS == 16 ? 8 : 1);
  __shared__ __align__(16) float slots[kTeamSlots];
  Team2 team;
  team.make(p.warps, slots, kTeamSlots);
  const int lane = threadIdx.x % 32;
  const int teams = blockDim.x / 32 / team.warps;
  const int tid = team.warp * 32 + lane;
  const int d2 = p.d / 2;
  const int per_head = p.d / (8 * VECS);   // items of a head
  const int items = p.H * per_head;
  const int nweights = p.norm == kRopeNormNone ? 0 : p.norm == kRopeNormToken ? p.H * p.d : p.d;
  const int tensors = p.staged;
  // shared memory: weights of q and k as two planes each (the first and the
  // last four channels of each vector), the teams' tables and sums, the stages
  const int nshared = p.shared_weights ? 2 * nweights : 0;
  float* weights = smem;
  float* table0 = smem + nshared + team.index * 2 * p.team_floats;
  uint8_t* ring = reinterpret_cast<uint8_t*>(smem + nshared + teams * 2 * p.team_floats) +
                  (threadIdx.x / 32) * p.depth * tensors * kTensor;

  const int first = team.warp * 32 * N + lane;   // this thread's items: first, first + 32, ...
  int chan[N];                                   // first channel of an item within its head
  unsigned place[N];                             // of an item in a token's output, by 8 elements
  bool on[N];
  const unsigned head_place = static_cast<unsigned>(p.L) * (p.d / 8);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int u = first + i * 32;
    on[i] = u < items;
    chan[i] = (u % per_head) * 8;
    place[i] = u / per_head * head_place + chan[i] / 8;
  }

  const unsigned L = p.L, tokens = p.B * L;   // below 2^31
  const unsigned step = gridDim.x * teams;
  unsigned next = blockIdx.x * teams + team.index;   // the token that the next copies bring
  auto load = [&](int stage) {
    if (next < tokens) {
      const int b = next / L;
      const int l = next - b * L;
      const uint32_t dst = smem_u32(ring + stage * tensors * kTensor) + lane * 16;
#pragma unroll
      for (int w = 0; w < 3; ++w) {
        const RopeTensor& x = w == 0 ? p.q : w == 1 ? p.k : p.v;
        if (w == 2 && p.staged < 3) continue;
        const T* in = static_cast<const T*>(x.in) + b * x.sb + l * x.sl;
        const uint32_t to = dst + w * kTensor;
        if (!HALF && p.packed) {
          // a token's vectors lie one after the other
          const uint8_t* from = reinterpret_cast<const uint8_t*>(in) + static_cast<long long>(team.warp) * kTensor + lane * 16;
          const int left = p.H * p.d * static_cast<int>(sizeof(T)) - team.warp * kTensor - lane * 16;
#pragma unroll
          for (int i = 0; i < N * kPieces; ++i)
            if (512 * i < left) cp_async_16(to + 512 * i, from + 512 * i);
        } else {
          // piece by piece: of vector v of item u, 16-byte pieces in address order
#pragma unroll
          for (int i = 0; i < N; ++i)
#pragma unroll
            for (int v = 0; v < VECS; ++v)
#pragma unroll
              for (int h = 0; h < kPieces; ++h) {
                const int at = lane + 32 * h;
                const int u = team.warp * 32 * N + i * 32 + at / kPieces;
                if (u < items)
                  cp_async_16(to + ((i * VECS + v) * kPieces + h) * 512,
                              in + (u / per_head) * x.sh + (u % per_head) * 8 + v * d2 + (at % kPieces) * 4);
              }
        }
      }
      next += step;
    }
    cp_async_commit();   // also where there is nothing to copy: groups are counted
  };
  unsigned tok = next;
  for (int s = 0; s < p.depth; ++s) load(s);

  for (int i = threadIdx.x; i < d2; i += blockDim.x) turns[i] = p.turns[i];
  for (int i = threadIdx.x; i < nshared / 8; i += blockDim.x) {
    const bool k = i >= nweights / 8;
    const RopeTensor& x = k ? p.k : p.q;
    const int v = k ? i - nweights / 8 : i;
    float f[1][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[0][j] = 1.f;
    if (x.weight) load_params<8, 1>(x.weight, x.weight_dtype, 0, v * 8, 0, INT_MAX, f);
    float4* plane = reinterpret_cast<float4*>(weights + (k ? nweights : 0));
    plane[v] = make_float4(f[0][0], f[0][1], f[0][2], f[0][3]);
    plane[nweights / 8 + v] = make_float4(f[0][4], f[0][5], f[0][6], f[0][7]);
  }
  __syncthreads();

  int stage = 0, parity = 0;
  for (; tok < tokens; tok += step) {
    const int b = tok / L;
    const int l = tok - b * L;
    float* table = table0 + parity * p.team_floats;
    float* sums = table + p.d;
    parity ^= 1;
    for (int i = tid; i < d2; i += team.warps * 32) {
      const double t = rope_position(p, b, l, p.axis[i]) * turns[i];
      float sn, cs;
      sincospif(2.f * static_cast<float>(t - rint(t)), &sn, &cs);
      table[i] = cs;
      table[d2 + i] = sn;
    }
    // all but the depth - 1 youngest groups are complete: this token has come
    if (p.depth == 1) cp_async_wait<0>();
    else if (p.depth == 2) cp_async_wait<1>();
    else if (p.depth == 3) cp_async_wait<2>();
    else cp_async_wait<3>();
    __syncwarp();
    const uint8_t* src = ring + stage * tensors * kTensor;

    float m[2][N];   // 1 / rms of q and of k, for each item
    if (p.norm != kRopeNormNone) {
      float total[2] = {0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 2; ++w) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float2 s = make_float2(0.f, 0.f);
          if (on[i]) {
#pragma unroll
            for (int v = 0; v < VECS; ++v) {
              float a[8];
              take_staged<T>(src + w * kTensor, (i * VECS + v) * 32 + lane, a);
              sum_sq<8>(s, a);
            }
          }
          m[w][i] = s.x + s.y;
          total[w] += m[w][i];
        }
      }
      if (p.norm == kRopeNormToken) {
        team.template sum<2>(total);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const float r = rsqrtf(fmaf(total[w], p.inv_channels, p.eps));
#pragma unroll
          for (int i = 0; i < N; ++i) m[w][i] = r;
        }
      } else if (p.by_lanes) {
        // a head's items lie in neighbouring lanes of one warp
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int i = 0; i < N; ++i) {
            for (int o = per_head / 2; o; o >>= 1) m[w][i] += __shfl_xor_sync(0xFFFFFFFFu, m[w][i], o);
            m[w][i] = rsqrtf(fmaf(m[w][i], p.inv_channels, p.eps));
          }
        team.sync();   // the table is complete
      } else {
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (on[i]) sums[w * items + first + i * 32] = m[w][i];
        team.sync();   // so are the table and the sums
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int i = 0; i < N; ++i) {
            if (!on[i]) continue;
            const float* s = sums + w * items + (first + i * 32) / per_head * per_head;
            float r = 0.f;
            for (int j = 0; j < per_head; ++j) r += s[j];
            m[w][i] = rsqrtf(fmaf(r, p.inv_channels, p.eps));
          }
      }
    } else {
      team.sync();   // the table is complete
    }

    const long long out0 = (static_cast<long long>(b) * p.H * L + l) * p.d;
    T* const outs[3] = {static_cast<T*>(p.q.out) + out0, static_cast<T*>(p.k.out) + out0, static_cast<T*>(p.v.out) + out0};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!on[i]) continue;
      const long long o = static_cast<long long>(place[i]) * 8;
      float cs[8], sn[8];
      float4 c4, s4;
      if constexpr (HALF) {
#pragma unroll
        for (int j = 0; j < 8; ++j) cs[j] = table[chan[i] + j], sn[j] = table[d2 + chan[i] + j];
      } else {
        c4 = *reinterpret_cast<const float4*>(table + chan[i] / 2);
        s4 = *reinterpret_cast<const float4*>(table + d2 + chan[i] / 2);
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        float a[VECS][8];
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
          take_staged<T>(src + w * kTensor, (i * VECS + v) * 32 + lane, a[v]);
          if (nweights) {
            int at = chan[i] / 8 + v * (d2 / 8);   // the vector's weights
            if (p.norm == kRopeNormToken) at += (first + i * 32) / per_head * (p.d / 8);
            mul_s<8>(a[v], m[w][i]);
            if (p.shared_weights) {
              const float4* plane = reinterpret_cast<const float4*>(weights + w * nweights);
              const float4 g = plane[at], h = plane[nweights / 8 + at];
              const float f[8] = {g.x, g.y, g.z, g.w, h.x, h.y, h.z, h.w};
              mul_v<8>(a[v], f);
            } else {
              const RopeTensor& x = w ? p.k : p.q;
              float f[1][8];
              if (x.weight) {
                load_params<8, 1>(x.weight, x.weight_dtype, 0, at * 8, 0, INT_MAX, f);
                mul_v<8>(a[v], f[0]);
              }
            }
          }
        }
        if constexpr (HALF) rope_turn_half(a[0], a[1], cs, sn);
        else rope_turn(a[0], c4, s4);
#pragma unroll
        for (int v = 0; v < VECS; ++v) store_row(outs[w] + o + v * d2, a[v]);
      }
      if (p.v.in) {
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
          Raw<T, 8> r;
          if (p.staged < 3) {
            load_raw(r, static_cast<const T*>(p.v.in) + b * p.v.sb + l * p.v.sl + (first + i * 32) / per_head * p.v.sh + chan[i] + v * d2);
          } else {
#pragma unroll
            for (int h = 0; h < kPieces; ++h)
              r.r[h] = *reinterpret_cast<const uint4*>(src + 2 * kTensor + ((i * VECS + v) * 32 + lane) * 8 * sizeof(T) + 16 * h);
          }
          store_raw(outs[2] + o + v * d2, r);
        }
      }
    }
    __syncwarp();   // all lanes have read the stage
    load(stage);
    stage = stage + 1 == p.depth ? 0 : stage + 1;
  }
  cp_async_wait<0>();
}

}  // namespace solattn
