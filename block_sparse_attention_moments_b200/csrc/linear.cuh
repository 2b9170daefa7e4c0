// linear.cuh — products of 8-bit integers with a scale for each token and each
// output channel:
//   y[m, n] = (sum_k a[m, k] w[n, k]) * a_scale[m] * w_scale[n] + bias[n]
// The sum is exact: s8 x s8 products accumulate in s32 (tcgen05.mma kind::i8),
// which holds K up to 131071 (128 * 128 * K < 2^31).
//
// linear_kernel: persistent, warp-specialised.  A pair of CTAs (cta_group::2)
// works on a tile of 256 tokens x BN channels, a single CTA (cta_group::1) on
// 128 x BN.  Warp 0 copies A and W tiles of 128 bytes of K by TMA into a ring
// of stages, warp 1 issues the MMAs, warps 2-5 read the accumulators from TMEM
// and write the output; two accumulators alternate, so that one tile's output
// is written while the next one's products run.
#pragma once

#include "rows.cuh"
#include "sm100_ptx.cuh"

namespace solattn {

constexpr int kLinThreads = 192;
constexpr int kLinStageA = 128 * 128;                    // bytes of A of a stage (of a CTA)
constexpr uint64_t kLinTimeoutNs = 2000000000ull;

// Set by a kernel whose wait gave up; read by sol_attn_linear_status.
static __device__ unsigned g_linear_status;

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
};

template <int CG, int BN>
struct LinearConfig {
  static constexpr int kStageB = BN / CG * 128;
  static constexpr int kStage = kLinStageA + kStageB;
  static constexpr int kOut = 4 * 2 * 4096;              // per epilogue warp two buffers of 32 rows x 128 bytes
  static constexpr int kStages = (224 * 1024 - kOut) / kStage > 8 ? 8 : (224 * 1024 - kOut) / kStage;
  static constexpr int kTmem = 2 * BN < 32 ? 32 : 2 * BN;
  static constexpr size_t kSmem = static_cast<size_t>(kStages) * kStage + kOut + 1024 + 512;
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

__device__ __forceinline__ void linear_tile(const LinearParams& p, int t, int* m, int* n) {
  const int per_band = p.band * p.tiles_n;
  const int b = t / per_band, r = t - b * per_band;
  const int rows = min(p.band, p.tiles_m - b * p.band);   // the last band may be narrower
  *n = r / rows;
  *m = b * p.band + (r - *n * rows);
}

template <int CG, int BN, typename T>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                  const __grid_constant__ CUtensorMap map_out, const __grid_constant__ LinearParams p) {
  using C = LinearConfig<CG, BN>;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* out_buf = base + C::kStages * C::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(out_buf + C::kOut);
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
      mbar_init(&acc_empty[i], 4 * CG);   // the epilogue warps of the tile's CTAs
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

  if (warp == 0 && lane == 0) {
    int it = 0;
    for (int t = first; t < tiles && ok; t += step) {
      int tm, tn;
      linear_tile(p, t, &tm, &tn);
      const int row_a = (tm * CG + rank) * 128;
      const int row_w = tn * BN + rank * (BN / CG);
      for (int k = 0; k < kblocks; ++k, ++it) {
        const int s = it % C::kStages;
        if (!mbar_wait(&empty[s], ((it / C::kStages) & 1) ^ 1, abort, kLinTimeoutNs)) { ok = false; break; }
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
      if (!mbar_wait(&acc_empty[buf], ((tile >> 1) & 1) ^ 1, abort, kLinTimeoutNs)) { ok = false; break; }
      tc_fence_after();
      const uint32_t d = tmem + buf * BN;
      for (int k = 0; k < kblocks; ++k, ++it) {
        const int s = it % C::kStages;
        if (!mbar_wait(&full[s], (it / C::kStages) & 1, abort, kLinTimeoutNs)) { ok = false; break; }
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
    const int q = warp & 3;                 // the TMEM lanes that this warp may read
    uint8_t* stage_out = out_buf + q * 2 * 4096;
    constexpr int kCols = 128 / sizeof(T);  // channels of a 128-byte row of the output buffer
    int tile = 0, chunk = 0;
    for (int t = first; t < tiles && ok; t += step, ++tile) {
      int tm, tn;
      linear_tile(p, t, &tm, &tn);
      const int buf = tile & 1;
      const int row0 = (tm * CG + static_cast<int>(rank)) * 128 + q * 32;
      const int row = row0 + lane;
      const float sa = row < p.M ? p.a_scale[row] : 0.f;
      ok = mbar_wait(&acc_full[buf], (tile >> 1) & 1, abort, kLinTimeoutNs);
      if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
      tc_fence_after();
      const uint32_t src = tmem + buf * BN + (static_cast<uint32_t>(q * 32) << 16);
      for (int c0 = 0; c0 < BN; c0 += kCols) {
        const int col0 = tn * BN + c0;
        const bool last = c0 + kCols >= BN;
        uint8_t* sbuf = stage_out + (chunk & 1) * 4096;
        uint32_t r[kCols];
#pragma unroll
        for (int j = 0; j < kCols; j += 32) tmem_ld_x32f(src + c0 + j, reinterpret_cast<float*>(r) + j);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < kCols; j += 32) reg_fence32(reinterpret_cast<float*>(r) + j);
        if (last) {   // the accumulator has been read
          tc_fence_before();
          if (lane == 0) {
            if constexpr (CG == 2) mbar_arrive_remote(map_to_rank(smem_u32(&acc_empty[buf]), 0));
            else mbar_arrive(&acc_empty[buf]);
          }
        }
        if (col0 >= p.N || row0 >= p.M) continue;
        ++chunk;
        // the TMA store of this buffer two chunks ago has read it
        if (!p.direct) {
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kCols; j += 16 / sizeof(T)) {
          float f[16 / sizeof(T)];
#pragma unroll
          for (int i = 0; i < static_cast<int>(16 / sizeof(T)); ++i) {
            const int n = min(col0 + j + i, p.N - 1);
            f[i] = fmaf(static_cast<float>(static_cast<int>(r[j + i])) * sa, p.w_scale[n], bias_at(p, n));
          }
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
          for (int i = 0; i < rows; ++i) {
            T* o = static_cast<T*>(p.out) + (row0 + i) * p.out_pitch + col0;
            for (int j = lane; j < cols; j += 32) {
              const int byte = j * static_cast<int>(sizeof(T));
              o[j] = *reinterpret_cast<const T*>(sbuf + i * 128 + (((byte >> 4) ^ (i & 7)) << 4) + (byte & 15));
            }
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

}  // namespace solattn
