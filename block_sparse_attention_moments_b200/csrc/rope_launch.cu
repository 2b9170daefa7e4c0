// rope_launch.cu — launches of the rotary kernel.
#include <algorithm>

#include "host.h"
#include "layer_launch.h"

namespace solattn {
namespace {

constexpr size_t kRopeShared = 220 * 1024;       // shared memory of the rotary kernel

template <typename T, bool HALF, int WARPS>
int launch_rope_as(RopeParams p, int dev, int sms, cudaStream_t st) {
  const int items = p.H * p.d / (HALF ? 16 : 8);
  const int group = p.d / (HALF ? 16 : 8);
  p.by_lanes = 32 % group == 0;
  // per team and parity: cosines and sines, and the items' sums where lanes cannot add them
  p.team_floats = p.d + (p.norm == kRopeNormHead && !p.by_lanes ? (2 * items + 3) / 4 * 4 : 0);
  const size_t tables = 2 * p.team_floats * sizeof(float), part = static_cast<size_t>(p.warps) * kRopeVectors * 32 * 8 * sizeof(T);
  // the widest fp32 rows leave no room for v, and less than that for the weights of a token norm
  p.staged = p.v.in && tables + 3 * part <= kRopeShared ? 3 : 2;
  const size_t stage = p.staged * part, per_team = tables + stage;
  size_t weights = p.norm == kRopeNormNone ? 0 : (p.norm == kRopeNormToken ? p.H : 1) * p.d * 2 * sizeof(float);
  p.shared_weights = weights + per_team <= kRopeShared;
  if (!p.shared_weights) weights = 0;
  int teams = p.warps > 1 ? std::min(15, kRopeThreads / 32 / p.warps) : kRopeThreads / 32;
  teams = std::max(1, std::min<int>(teams, static_cast<int>((kRopeShared - weights) / per_team)));
  p.depth = 1;
  while (p.depth < 4 && weights + teams * (per_team + p.depth * stage) <= kRopeShared) ++p.depth;
  const size_t smem = weights + teams * (2 * p.team_floats * sizeof(float) + p.depth * stage);
  static bool attr_set[kMaxDevices] = {false};   // the attribute is set per device
  if (!attr_set[dev]) {
    CUDA_TRY(cudaFuncSetAttribute(rope_kernel<T, HALF, WARPS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  static_cast<int>(kRopeShared)));
    attr_set[dev] = true;
  }
  const long long tokens = static_cast<long long>(p.B) * p.L;
  const int grid = static_cast<int>(std::min<long long>((tokens + teams - 1) / teams, sms));
  rope_kernel<T, HALF, WARPS><<<grid, teams * p.warps * 32, smem, st>>>(p);
  CUDA_TRY(cudaGetLastError());
  return SOL_ATTN_OK;
}

template <typename T, bool HALF>
int launch_rope_warps(RopeParams p, int dev, int sms, cudaStream_t st) {
  const int per_warp = 32 * kRopeVectors * 8;
  p.warps = (p.H * p.d + per_warp - 1) / per_warp;
  if (p.warps == 1) return launch_rope_as<T, HALF, 1>(p, dev, sms, st);
  if (p.warps <= 8) return launch_rope_as<T, HALF, 8>(p, dev, sms, st);
  return launch_rope_as<T, HALF, 16>(p, dev, sms, st);
}

template <typename T>
int launch_rope_type(const RopeParams& p, int dev, int sms, cudaStream_t st) {
  return p.half ? launch_rope_warps<T, true>(p, dev, sms, st) : launch_rope_warps<T, false>(p, dev, sms, st);
}

}  // namespace

int launch_rope(const RopeParams& p, int dtype, int dev, int sms, cudaStream_t st) {
  if (dtype == SOL_ATTN_BF16) return launch_rope_type<__nv_bfloat16>(p, dev, sms, st);
  if (dtype == SOL_ATTN_FP16) return launch_rope_type<__half>(p, dev, sms, st);
  return launch_rope_type<float>(p, dev, sms, st);
}

}  // namespace solattn
