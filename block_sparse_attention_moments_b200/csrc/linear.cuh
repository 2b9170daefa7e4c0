// linear.cuh — products of 8-bit integers with a scale for each token and each
// output channel:
//   y[m, n] = (sum_k a[m, k] w[n, k]) * a_scale[m] * w_scale[n] + bias[n]
// The sum is exact: s8 x s8 products accumulate in s32 (tcgen05.mma kind::i8),
// which holds K up to 131071 (128 * 128 * K < 2^31).
//
// linear_kernel: persistent, warp-specialised.  A pair of CTAs (cta_group::2)
// works on a tile of 256 tokens x BN channels, a single CTA (cta_group::1) on
// 128 x BN.  Warp 0 copies A and W tiles of 128 bytes of K by TMA into a ring
// of stages, warp 1 issues the MMAs, warps 2-9 read the accumulators from TMEM
// and write the output; two accumulators alternate, so that one tile's output
// is written while the next one's products run.
//
// Measured (B200): 75600 x 15360 x 5120 with bf16 output 4.31 to 4.51 ms back to
// back for seconds, 2.64 to 2.76 POP/s, where the power limit lowers the clock
// (twice the measured sustained bf16 rate is 2.77); with pauses between calls 3.64
// to 3.80 ms, 3.13 to 3.27 POP/s (twice the burst rate is 3.26).  16384 x 5120 x
// 5120 270 us.  Shorter K (16384 x 1024 x 1024: 20 to 23 us for 10.5) has 256 tiles
// for 74 pairs, 3.5 waves that take four, and eight steps a tile, in each of which
// an SM is brought 32 KB of operands from L2.
#pragma once

#include "rows.cuh"
#include "sm100_ptx.cuh"

namespace solattn {

constexpr int kLinThreads = 320;    // copies, MMAs, and eight warps for the output
constexpr int kFewThreads = 192;
constexpr int kLinStageA = 128 * 128;                    // bytes of A of a stage (of a CTA)

// Set by a kernel whose wait gave up (1) or whose shared memory lies at another
// alignment than the tiles' swizzle needs (2); read by sol_attn_linear_status.
static __device__ unsigned g_linear_status;

__device__ __forceinline__ bool tiles_aligned(const void* base) {
  if ((smem_u32(base) & 1023) == 0) return true;
  atomicOr(&g_linear_status, 2u);
  return false;
}

struct LinearParams {
  int M, N, K;
  int tiles_m, tiles_n, band;   // tiles go through bands of `band` tiles of M, M fastest
  const float* a_scale;
  const float* w_scale;
  const void* bias;             // null: none
  int bias_dtype;
  void* out;
  long long out_pitch;          // elements
  int direct;                   // the output's rows are not aligned for TMA
  int stall;                    // test of the waits' limits: nothing is copied
  unsigned long long timeout_ns;
};

template <int CG, int BN>
struct LinearConfig {
  static constexpr int kStageB = BN / CG * 128;
  static constexpr int kStage = kLinStageA + kStageB;
  static constexpr int kOut = 8 * 4096;                  // per output warp 32 rows x 128 bytes
  static constexpr int kStages = (224 * 1024 - kOut) / kStage;
  static constexpr int kTmem = 2 * BN;                   // columns of two accumulators
  static constexpr int kParams = BN * 8;                 // the tile's scales and biases, fp32
  static constexpr size_t kSmem = static_cast<size_t>(kStages) * kStage + kOut + kParams + 512;
  static_assert(kSmem <= 227 * 1024, "shared memory of a block");
};

// kind::i8 instruction descriptor: D s32 (2), A and B s8 (1), both K-major.
__host__ __device__ constexpr uint32_t idesc_s8_s32(uint32_t M, uint32_t N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

template <int CG>
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  if constexpr (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, %4}], [%2];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1)
               : "memory");
}

template <int CG>
__device__ __forceinline__ void umma_s8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (CG == 1)
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
                 : "memory");
  else
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
                 : "memory");
}
// Arrives on the barrier (of both CTAs of a pair) when the MMAs issued so far are complete.
template <int CG>
__device__ __forceinline__ void umma_commit_all(uint64_t* bar) {
  if constexpr (CG == 1)
    umma_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_alloc_all(uint32_t* dst, uint32_t cols) {
  if constexpr (CG == 1) {
    tmem_alloc(dst, cols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc_all(uint32_t addr, uint32_t cols) {
  if constexpr (CG == 1) tmem_dealloc(addr, cols);
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

__device__ __forceinline__ float bias_at(const LinearParams& p, int n) {
  float f[1][1] = {{0.f}};
  if (p.bias) load_params<1, 1>(p.bias, p.bias_dtype, n, 0, 0, 1, f);
  return f[0][0];
}

// One output value; every kernel here forms it this way, so that a token's
// output does not depend on the number of tokens beside it.
__device__ __forceinline__ float linear_value(int sum, float a_scale, float w_scale, float bias) {
  return fmaf(__fmul_rn(__int2float_rn(sum), a_scale), w_scale, bias);
}
// The same for four channels of a token.
__device__ __forceinline__ void linear_values4(const uint32_t* sum, float a_scale, const float4& w, const float4& b, float* f) {
  const float2 s = make_float2(a_scale, a_scale);
  const float2 x = __fmul2_rn(make_float2(__int2float_rn(sum[0]), __int2float_rn(sum[1])), s);
  const float2 y = __fmul2_rn(make_float2(__int2float_rn(sum[2]), __int2float_rn(sum[3])), s);
  const float2 u = __ffma2_rn(x, make_float2(w.x, w.y), make_float2(b.x, b.y));
  const float2 v = __ffma2_rn(y, make_float2(w.z, w.w), make_float2(b.z, b.w));
  f[0] = u.x, f[1] = u.y, f[2] = v.x, f[3] = v.y;
}

__device__ __forceinline__ void linear_tile(const LinearParams& p, int t, int* m, int* n) {
  const int per_band = p.band * p.tiles_n;
  const int b = t / per_band, r = t - b * per_band;
  const int rows = min(p.band, p.tiles_m - b * p.band);   // the last band may be narrower
  *n = r / rows;
  *m = b * p.band + (r - *n * rows);
}

// Barrier 1 of the eight output warps; whether all of their threads are well.
__device__ __forceinline__ bool all_of_epilogue(bool ok) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(r)
               : "r"(static_cast<uint32_t>(ok))
               : "memory");
  return r != 0;
}

template <int CG, int BN, typename T>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                  const __grid_constant__ CUtensorMap map_out, const __grid_constant__ LinearParams p) {
  using C = LinearConfig<CG, BN>;
  extern __shared__ __align__(1024) uint8_t base[];
  if (!tiles_aligned(base)) return;
  uint8_t* out_buf = base + C::kStages * C::kStage;
  float* params = reinterpret_cast<float*>(out_buf + C::kOut);   // scales, then biases, of the tile's channels
  uint64_t* full = reinterpret_cast<uint64_t*>(params + 2 * BN);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 8 * CG);   // the output warps of the tile's CTAs
    }
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_all<CG>(tmem_slot, C::kTmem);
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int tiles = p.tiles_m * p.tiles_n;
  const int first = blockIdx.x / CG, step = gridDim.x / CG;
  const int kblocks = (p.K + 127) / 128;
  bool ok = true;

  if (warp == 0 && lane == 0 && !p.stall) {
    int it = 0;
    for (int t = first; t < tiles && ok; t += step) {
      int tm, tn;
      linear_tile(p, t, &tm, &tn);
      const int row_a = (tm * CG + rank) * 128;
      const int row_w = tn * BN + rank * (BN / CG);
      for (int k = 0; k < kblocks; ++k, ++it) {
        const int s = it % C::kStages;
        if (!mbar_wait(&empty[s], ((it / C::kStages) & 1) ^ 1, abort, p.timeout_ns)) { ok = false; break; }
        if (rank == 0) mbar_arrive_expect_tx(&full[s], CG * C::kStage);
        uint32_t bar = smem_u32(&full[s]);
        if constexpr (CG == 2) bar = map_to_rank(bar, 0);
        const uint32_t dst = smem_u32(base + s * C::kStage);
        tma_load_2d<CG>(dst, &map_a, bar, k * 128, row_a);
        tma_load_2d<CG>(dst + kLinStageA, &map_w, bar, k * 128, row_w);
      }
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    constexpr uint32_t idesc = idesc_s8_s32(128 * CG, BN);
    int it = 0, tile = 0;
    for (int t = first; t < tiles && ok; t += step, ++tile) {
      const int buf = tile & 1;
      if (!mbar_wait(&acc_empty[buf], ((tile >> 1) & 1) ^ 1, abort, p.timeout_ns)) { ok = false; break; }
      tc_fence_after();
      const uint32_t d = tmem + buf * BN;
      for (int k = 0; k < kblocks; ++k, ++it) {
        const int s = it % C::kStages;
        if (!mbar_wait(&full[s], (it / C::kStages) & 1, abort, p.timeout_ns)) { ok = false; break; }
        tc_fence_after();
        const uint32_t sa = smem_u32(base + s * C::kStage);
        const uint64_t da = sdesc_sw128(sa, 16, 1024), db = sdesc_sw128(sa + kLinStageA, 16, 1024);
#pragma unroll
        for (int j = 0; j < 4; ++j)   // 32 bytes of K each: the start address moves within the swizzled rows
          umma_s8<CG>(d, da + 2 * j, db + 2 * j, idesc, (k | j) != 0);
        umma_commit_all<CG>(&empty[s]);
      }
      if (ok) umma_commit_all<CG>(&acc_full[buf]);
    }
  } else if (warp >= 2) {
    // Two warps to each quarter of the TMEM lanes (a warp may read the quarter
    // of its number), every other chunk of columns each: one warp's conversions
    // and stores fill the other's waits.
    const int q = warp & 3, half = (warp - 2) >> 2;
    uint8_t* sbuf = out_buf + (warp - 2) * 4096;
    constexpr int kCols = 128 / sizeof(T);  // channels of a 128-byte row of the output buffer
    int tile = 0;
    for (int t = first; t < tiles; t += step, ++tile) {
      int tm, tn;
      linear_tile(p, t, &tm, &tn);
      const int buf = tile & 1;
      const int row0 = (tm * CG + static_cast<int>(rank)) * 128 + q * 32;
      const int row = row0 + lane;
      const float sa = row < p.M ? p.a_scale[row] : 0.f;
      // the channels' scales and biases, fetched while the tile is being multiplied
      const int c = threadIdx.x - 64;
      const bool there = c < BN && tn * BN + c < p.N;
      const float scale = there ? p.w_scale[tn * BN + c] : 0.f, bias = there ? bias_at(p, tn * BN + c) : 0.f;
      // Those of the tile before have been read.  A warp whose wait gave up
      // says so here, where all leave together: none is left at a barrier.
      ok = all_of_epilogue(ok);
      if (!ok) break;
      if (c < BN) params[c] = scale, params[BN + c] = bias;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      ok = mbar_wait(&acc_full[buf], (tile >> 1) & 1, abort, p.timeout_ns);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) continue;
      tc_fence_after();
      const uint32_t src = tmem + buf * BN + (static_cast<uint32_t>(q * 32) << 16);
      static_assert(BN % (2 * kCols) == 0, "both warps of a quarter have as many chunks");
      const int last = BN - (2 - half) * kCols;
      for (int c0 = half * kCols; c0 < BN; c0 += 2 * kCols) {
        const int col0 = tn * BN + c0;
        uint32_t r[kCols];
#pragma unroll
        for (int j = 0; j < kCols; j += 32) tmem_ld_x32f(src + c0 + j, reinterpret_cast<float*>(r) + j);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < kCols; j += 32) reg_fence32(reinterpret_cast<float*>(r) + j);
        if (c0 == last) {   // this warp has read its part of the accumulator
          tc_fence_before();
          if (lane == 0) {
            if constexpr (CG == 2) mbar_arrive_remote(map_to_rank(smem_u32(&acc_empty[buf]), 0));
            else mbar_arrive(&acc_empty[buf]);
          }
        }
        if (col0 >= p.N || row0 >= p.M) continue;
        // the store of the chunk before has read the buffer
        if (!p.direct) {
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kCols; j += 16 / sizeof(T)) {
          float f[16 / sizeof(T)];
#pragma unroll
          for (int i = 0; i < static_cast<int>(16 / sizeof(T)); i += 4)
            linear_values4(r + j + i, sa, *reinterpret_cast<const float4*>(params + c0 + j + i),
                           *reinterpret_cast<const float4*>(params + BN + c0 + j + i), f + i);
          uint4 w;
          if constexpr (sizeof(T) == 2)
            w = make_uint4(narrow2<T>(f[0], f[1]), narrow2<T>(f[2], f[3]), narrow2<T>(f[4], f[5]), narrow2<T>(f[6], f[7]));
          else
            w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
          const int piece = j * static_cast<int>(sizeof(T)) / 16;
          *reinterpret_cast<uint4*>(sbuf + lane * 128 + ((piece ^ (lane & 7)) << 4)) = w;
        }
        if (!p.direct) {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&map_out, smem_u32(sbuf), col0, row0);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        } else {
          __syncwarp();
          const int rows = min(32, p.M - row0), cols = min(kCols, p.N - col0);
          T* o = static_cast<T*>(p.out) + row0 * p.out_pitch + col0;
#pragma unroll
          for (int j0 = 0; j0 < kCols; j0 += 32) {
            const int byte = (j0 + lane) * static_cast<int>(sizeof(T));
#pragma unroll 8
            for (int i = 0; i < 32; ++i)
              if (i < rows && j0 + lane < cols)
                o[i * p.out_pitch + j0 + lane] =
                    *reinterpret_cast<const T*>(sbuf + i * 128 + (((byte >> 4) ^ (i & 7)) << 4) + (byte & 15));
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  if (!ok) {
    // a wait gave up: say so, stop the other roles, and let copies in flight land
    *abort = 1;
    atomicOr(&g_linear_status, 1u);
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) {}
  }
  __syncwarp();
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_all<CG>(tmem, C::kTmem);
}


// ------------------------------------------------------------------ one to four tokens
// The weights are read once and each of their bytes meets MT tokens: bound by
// their bytes, so plain 16-byte loads and dp4a.  A warp takes R channels, its
// lanes 16 bytes each of K a step; where there are few channels the block's
// warps share them and split K.  2 x 30720 x 5120: 28.6 us (24.0 at the copy
// rate); 1 x 5120 x 5120 5.8 us (4.0); 4 x 15360 x 5120 16.1 us, the MMA form
// below 13.3, but 8.8 against 8.3 at 5120 channels and 5.1 against 4.1 at 256.
constexpr int kVecRows = 4;      // channels of a warp
constexpr int kVecWarps = 4;     // warps of a block

struct LinearVecParams {
  LinearParams p;
  const int8_t* a;
  long long a_pitch;
  const int8_t* w;
  long long w_pitch;
  int split;      // warps that share channels: 1 or kVecWarps
};

// 16 bytes of a row of K bytes at k; bytes past the row read as zero.
__device__ __forceinline__ int4 load_row16(const int8_t* row, int k, int K) {
  if (k + 16 <= K) {
    int4 r;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(row + k));
    return r;
  }
  int v[4] = {0, 0, 0, 0};
  for (int i = 0; k + i < K; ++i) v[i / 4] |= (row[k + i] & 255) << (8 * (i % 4));
  return make_int4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ int dot16(const int4& a, const int4& b, int s) {
  return __dp4a(a.w, b.w, __dp4a(a.z, b.z, __dp4a(a.y, b.y, __dp4a(a.x, b.x, s))));
}

template <int MT, typename T>
__global__ void __launch_bounds__(kVecWarps * 32) linear_vec_kernel(const __grid_constant__ LinearVecParams v) {
  __shared__ int part[kVecWarps][kVecRows * MT];
  const LinearParams& p = v.p;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int sub = warp % v.split;   // this warp's share of K
  const int n0 = (blockIdx.x * (kVecWarps / v.split) + warp / v.split) * kVecRows;
  int acc[kVecRows][MT];
#pragma unroll
  for (int r = 0; r < kVecRows; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = 0;
  const int8_t* w[kVecRows];
#pragma unroll
  for (int r = 0; r < kVecRows; ++r) w[r] = v.w + static_cast<long long>(min(n0 + r, p.N - 1)) * v.w_pitch;
  constexpr int U = MT <= 2 ? 2 : 1;   // steps under way together
  for (int k = (sub * 32 + lane) * 16; k < p.K; k += U * v.split * 512) {
    int4 x[U][kVecRows], y[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int ku = k + u * v.split * 512;
#pragma unroll
      for (int r = 0; r < kVecRows; ++r) x[u][r] = ku < p.K ? load_row16(w[r], ku, p.K) : make_int4(0, 0, 0, 0);
#pragma unroll
      for (int m = 0; m < MT; ++m)
        y[u][m] = ku < p.K && m < p.M ? (ku + 16 <= p.K ? *reinterpret_cast<const int4*>(v.a + m * v.a_pitch + ku)
                                                        : load_row16(v.a + m * v.a_pitch, ku, p.K))
                                      : make_int4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < kVecRows; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[r][m] = dot16(x[u][r], y[u][m], acc[r][m]);
  }
  int mine = 0;   // the sum of channel lane / MT and token lane % MT
#pragma unroll
  for (int r = 0; r < kVecRows; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int s = __reduce_add_sync(0xFFFFFFFFu, acc[r][m]);
      if (lane == r * MT + m) mine = s;
    }
  if (v.split > 1) {
    if (lane < kVecRows * MT) part[warp][lane] = mine;
    __syncthreads();
    if (sub) return;
    if (lane < kVecRows * MT)
      for (int i = 1; i < v.split; ++i) mine += part[warp + i][lane];
  }
  const int n = n0 + lane / MT, m = lane % MT;
  if (lane < kVecRows * MT && n < p.N && m < p.M)
    static_cast<T*>(p.out)[m * p.out_pitch + n] = from_f32<T>(linear_value(mine, p.a_scale[m], p.w_scale[n], bias_at(p, n)));
}

// ------------------------------------------------------------------ few tokens
// The tile the other way round: 128 channels are the rows of the MMA and BT
// tokens its columns, so that the weights, which bound it, fill whole tiles
// (the tiles of further tokens find them in L2).  A cluster of `split` CTAs shares a tile's K; each reads its accumulators and
// gives every rank the sums of that rank's tokens through distributed shared
// memory, where the rank adds them in order.  One tile to a cluster, a few
// CTAs to an SM.  15360 x 5120: 16 tokens 13.0 us (12.1 at the copy rate), 64
// 17.8, 128 23.5.
template <int BT>
struct FewConfig {
  static constexpr int kStage = kLinStageA + BT * 128;
  static constexpr int kStages = BT <= 32 ? 4 : 3;
  static constexpr int kParts = BT * 128 * 4;
  static constexpr size_t kSmem = static_cast<size_t>(kStages) * kStage + kParts + BT * 4 + 256;
};

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

template <int BT, typename T>
__global__ void __launch_bounds__(kFewThreads)
    linear_few_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                      const __grid_constant__ LinearParams p, int log_split) {
  using C = FewConfig<BT>;
  extern __shared__ __align__(1024) uint8_t base[];
  if (!tiles_aligned(base)) return;
  uint32_t* parts = reinterpret_cast<uint32_t*>(base + C::kStages * C::kStage);   // [split][BT / split][128]
  float* a_scale = reinterpret_cast<float*>(parts + BT * 128);
  uint64_t* full = reinterpret_cast<uint64_t*>(a_scale + BT);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  constexpr int kTmem = BT < 32 ? 32 : BT;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_rank();
  const int split = 1 << log_split, tile = blockIdx.x >> log_split;
  const int n0 = tile / p.tiles_m * 128, t0 = tile % p.tiles_m * BT;   // first channel and token
  const int tokens = p.M - t0;
  if (split > 1) cluster_arrive();   // met before the first access to another CTA's memory, which must have started
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(acc_full, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_all<1>(tmem_slot, kTmem);
  for (int i = threadIdx.x; i < BT; i += kFewThreads) a_scale[i] = i < tokens ? p.a_scale[t0 + i] : 0.f;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int kblocks = (p.K + 127) / 128;
  const int k0 = kblocks * rank / split, k1 = kblocks * (rank + 1) / split;   // never empty: split <= kblocks
  bool ok = true;
  if (warp == 0 && lane == 0 && !p.stall) {
    for (int k = k0; k < k1; ++k) {
      const int it = k - k0, s = it % C::kStages;
      if (!mbar_wait(&empty[s], ((it / C::kStages) & 1) ^ 1, abort, p.timeout_ns)) { ok = false; break; }
      mbar_arrive_expect_tx(&full[s], C::kStage);
      const uint32_t dst = smem_u32(base + s * C::kStage);
      tma_load_2d<1>(dst, &map_w, smem_u32(&full[s]), k * 128, n0);
      tma_load_2d<1>(dst + kLinStageA, &map_a, smem_u32(&full[s]), k * 128, t0);
    }
  } else if (warp == 1 && lane == 0) {
    constexpr uint32_t idesc = idesc_s8_s32(128, BT);
    for (int k = k0; k < k1; ++k) {
      const int it = k - k0, s = it % C::kStages;
      if (!mbar_wait(&full[s], (it / C::kStages) & 1, abort, p.timeout_ns)) { ok = false; break; }
      tc_fence_after();
      const uint32_t sw = smem_u32(base + s * C::kStage);
      const uint64_t dw = sdesc_sw128(sw, 16, 1024), da = sdesc_sw128(sw + kLinStageA, 16, 1024);
#pragma unroll
      for (int j = 0; j < 4; ++j) umma_s8<1>(tmem, dw + 2 * j, da + 2 * j, idesc, (it | j) != 0);
      umma_commit(&empty[s]);
    }
    if (ok) umma_commit(acc_full);
  }
  const int q = warp & 3, row = q * 32 + lane;   // of warps 2 to 5: this thread's channel of the tile
  const int n = n0 + row;
  const float ws = warp >= 2 && n < p.N ? p.w_scale[n] : 0.f, b = warp >= 2 && n < p.N ? bias_at(p, n) : 0.f;
  uint32_t r[BT];
  if (warp >= 2) {
    ok = mbar_wait(acc_full, 0, abort, p.timeout_ns);
    ok = __all_sync(0xFFFFFFFFu, ok);
    tc_fence_after();
    if (ok) {
      const uint32_t src = tmem + (static_cast<uint32_t>(q * 32) << 16);
      if constexpr (BT < 32) {
        tmem_ld_x16f(src, reinterpret_cast<float*>(r));
      } else {
#pragma unroll
        for (int j = 0; j < BT; j += 32) tmem_ld_x32f(src + j, reinterpret_cast<float*>(r) + j);
      }
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < BT; j += 16) reg_fence16(reinterpret_cast<float*>(r) + j);
    }
  }
  if (!ok) {
    *abort = 1;
    atomicOr(&g_linear_status, 1u);
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) {}
  }
  __syncwarp();
  if (split > 1) {
    const int each = BT >> log_split;   // tokens of a rank
    cluster_wait();
    if (warp >= 2) {
      const uint32_t mine = smem_u32(parts + (rank * each) * 128 + row);
#pragma unroll
      for (int j = 0; j < BT; ++j)   // each is a power of two
        st_cluster(map_to_rank(mine + (j & (each - 1)) * 512, j >> (31 - __clz(each))), r[j]);
    }
    cluster_sync();
    if (warp >= 2 && ok && n < p.N) {
      const int m0 = rank * each, count = min(each, tokens - m0);
      T* o = static_cast<T*>(p.out) + (t0 + m0) * p.out_pitch + n;
#pragma unroll 4
      for (int j = 0; j < count; ++j) {
        int sum = 0;
        for (int s = 0; s < split; ++s) sum += parts[(s * each + j) * 128 + row];
        o[j * p.out_pitch] = from_f32<T>(linear_value(sum, a_scale[m0 + j], ws, b));
      }
    }
  } else if (warp >= 2 && ok && n < p.N) {
    T* o = static_cast<T*>(p.out) + t0 * p.out_pitch + n;
#pragma unroll
    for (int j = 0; j < BT; ++j)
      if (j < tokens) o[j * p.out_pitch] = from_f32<T>(linear_value(r[j], a_scale[j], ws, b));
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_all<1>(tmem, kTmem);
}

}  // namespace solattn
