// norm_launch.cu — launches of the norm kernels for one pair of types; compiled
// once for each with SOLATTN_NORM_NAME, SOLATTN_NORM_X and SOLATTN_NORM_Y.
#include <algorithm>

#include "host.h"
#include "layer_launch.h"

namespace solattn {
namespace {

constexpr size_t kNormRingShared = 220 * 1024;   // shared memory of the ring kernel: factors and rows
// Rows of a block, and tokens of a group, from which the ring kernel is taken
// (us of norm_kernel and of it: 450 rows of 5120 bf16 7.9 and 6.7, of 1544 4.6
// and 5.5; 700 of 5120 9.1 and 7.1, of 1024 6.1 and 3.6; 4500 of 5120 37.7 and
// 21.5; 8000 rows in groups of 4 89 and 89, of 8 77 and 61).
constexpr int kNormRingRows = 4;
constexpr int kNormRingGroup = 8;
constexpr int kNormRingVectors = 4;              // vectors of 8 that a thread holds of a row

template <typename TX, typename TY, int V, int N, bool RES, int THREADS>
int launch_norm_as(NormParams p, int sms, cudaStream_t st) {
  const long long rows = static_cast<long long>(p.B) * p.L;
  const int per_warp = 32 * N * V;
  p.warps = (p.C + per_warp - 1) / per_warp;
  const int teams = std::max(1, 4 / p.warps);
  const int threads = teams * p.warps * 32;
  const int blocks = std::max(1, 1024 / threads) * sms;
  const int grid = static_cast<int>(std::min<long long>((rows + teams - 1) / teams, blocks));
  norm_kernel<TX, TY, V, N, RES, THREADS><<<grid, threads, 0, st>>>(p);
  CUDA_TRY(cudaGetLastError());
  return SOL_ATTN_OK;
}

template <typename TX, typename TY, int R, bool RES, bool FULL, int WARPS>
int launch_norm_ring(NormParams p, size_t factors, int dev, int sms, cudaStream_t st) {
  constexpr int N = kNormRingVectors;
  const int teams = p.warps > 1 ? std::min(15, kNormRingThreads / 32 / p.warps) : kNormRingThreads / 32;
  const size_t stage = R == 1 ? 0 : static_cast<size_t>(p.warps) * R * N * 32 * 8 * (sizeof(TX) + (RES ? sizeof(TY) : 0));
  const int fit = R == 1 ? teams : static_cast<int>((kNormRingShared - factors) / stage);   // stages of all teams
  const int used = std::min(teams, fit);
  p.depth = R == 1 ? 1 : std::min(4, fit / used);
  static bool attr_set[kMaxDevices] = {false};   // the attribute is set per device
  if (!attr_set[dev]) {
    CUDA_TRY(cudaFuncSetAttribute(norm_ring_kernel<TX, TY, R, N, RES, FULL, WARPS>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kNormRingShared)));
    attr_set[dev] = true;
  }
  norm_ring_kernel<TX, TY, R, N, RES, FULL, WARPS><<<sms, used * p.warps * 32, factors + used * p.depth * stage, st>>>(p);
  CUDA_TRY(cudaGetLastError());
  return SOL_ATTN_OK;
}

template <typename TX, typename TY, int R, bool RES, bool FULL>
int launch_norm_warps(const NormParams& p, size_t factors, int dev, int sms, cudaStream_t st) {
  return p.warps == 1 ? launch_norm_ring<TX, TY, R, RES, FULL, 1>(p, factors, dev, sms, st)
                      : launch_norm_ring<TX, TY, R, RES, FULL, 8>(p, factors, dev, sms, st);
}

template <typename TX, typename TY, bool RES>
int launch_norm(NormParams p, bool vec, bool wide, int dev, int sms, cudaStream_t st) {
  if (vec) {
    // many rows of long groups, whose factors leave room for two teams' rows
    const long long rows = static_cast<long long>(p.B) * p.L;
    const int per_warp = 32 * kNormRingVectors * 8;
    const size_t factors = static_cast<size_t>(RES ? 3 + (p.post_bias.p != nullptr) : 2) * p.C * sizeof(float);
    p.warps = (p.C + per_warp - 1) / per_warp;
    for (p.inner_shift = 0; (1 << p.inner_shift) < p.x_inner;) ++p.inner_shift;
    if (rows >= kNormRingRows * static_cast<long long>(sms) && p.group >= kNormRingGroup && p.warps <= 8 &&
        (p.x_inner == p.C || p.x_inner == 1 << p.inner_shift)) {
      const bool full = p.C % per_warp == 0;
      if constexpr (sizeof(TX) == 4) {
        if (factors <= kNormRingShared)
          return full ? launch_norm_warps<TX, TY, 1, RES, true>(p, factors, dev, sms, st)
                      : launch_norm_warps<TX, TY, 1, RES, false>(p, factors, dev, sms, st);
      } else {
        const size_t stage = static_cast<size_t>(p.warps) * 2 * kNormRingVectors * 32 * 8 * (sizeof(TX) + (RES ? sizeof(TY) : 0));
        if (full && wide && factors <= kNormRingShared)
          return launch_norm_warps<TX, TY, 1, RES, true>(p, factors, dev, sms, st);
        if (factors + 2 * stage <= kNormRingShared)
          return launch_norm_warps<TX, TY, 2, RES, false>(p, factors, dev, sms, st);
      }
    }
    if (p.C <= 2816) return launch_norm_as<TX, TY, 8, 1, RES, 352>(p, sms, st);
    if (p.C <= 5120) return launch_norm_as<TX, TY, 8, 1, RES, 640>(p, sms, st);
    if (p.C <= 8192) return launch_norm_as<TX, TY, 8, 2, RES, 512>(p, sms, st);
    return launch_norm_as<TX, TY, 8, 4, RES, 512>(p, sms, st);
  }
  if (p.C <= 1408) return launch_norm_as<TX, TY, 1, 4, RES, 352>(p, sms, st);
  if (p.C <= 2560) return launch_norm_as<TX, TY, 1, 4, RES, 640>(p, sms, st);
  if (p.C <= 8192) return launch_norm_as<TX, TY, 1, 16, RES, 512>(p, sms, st);
  return launch_norm_as<TX, TY, 1, 32, RES, 512>(p, sms, st);
}

template <typename TX, typename TY>
int launch_norm_res(const NormParams& p, bool vec, bool wide, int dev, int sms, cudaStream_t st) {
  return p.y ? launch_norm<TX, TY, true>(p, vec, wide, dev, sms, st) : launch_norm<TX, TY, false>(p, vec, wide, dev, sms, st);
}

}  // namespace

int SOLATTN_NORM_NAME(const NormParams& p, bool vec, bool wide, int dev, int sms, cudaStream_t st) {
  return launch_norm_res<SOLATTN_NORM_X, SOLATTN_NORM_Y>(p, vec, wide, dev, sms, st);
}

}  // namespace solattn
