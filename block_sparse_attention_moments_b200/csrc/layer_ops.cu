// layer_ops.cu — C ABI of the operators around the attention (declared in
// include/sol_attn.h): argument checks and launches of the norm, rotary and
// 8-bit product kernels.  They hold no workspace: every call reads its inputs
// and writes its outputs only, so calls on several streams, devices or
// captured graphs do not meet.
#include <algorithm>
#include <climits>
#include <cmath>
#include <numeric>
#include <type_traits>

#include "host.h"
#include "linear.cuh"
#include "norm.cuh"
#include "rope.cuh"

using namespace solattn;

namespace {

constexpr int kMaxC = 16384;
constexpr int kMaxLinearK = 131071;   // 128 * 128 * K < 2^31
constexpr size_t kNormRingShared = 220 * 1024;   // shared memory of the ring kernel: factors and rows
// Tokens up to which channels are the rows of the tile (15360 x 5120: 128 tokens
// in tiles of 64 23 us, in one tile of 128 rows 37; 5120 x 5120: 200 tokens 19
// against 16.6 the other way round).
constexpr int kFewTokens = 128;
constexpr int kNormRingLeast = 32;               // rows of a block, and of a group, from which it is taken
constexpr int kNormRingVectors = 4;              // vectors of 8 that a thread holds of a row
constexpr size_t kRopeShared = 220 * 1024;       // shared memory of the rotary kernel

size_t dtype_size(int dtype) { return dtype == SOL_ATTN_FP32 ? 4 : 2; }

bool dtype_ok(int dtype) { return dtype == SOL_ATTN_BF16 || dtype == SOL_ATTN_FP16 || dtype == SOL_ATTN_FP32; }

int sm_count(int dev, int* n) {
  static int cached[kMaxDevices] = {0};
  if (!cached[dev]) CUDA_TRY(cudaDeviceGetAttribute(&cached[dev], cudaDevAttrMultiProcessorCount, dev));
  *n = cached[dev];
  return SOL_ATTN_OK;
}

// The current device, checked, and its number of SMs.
int device(int* dev, int* sms) {
  int rc;
  if ((rc = current_device(dev)) || (rc = check_arch(*dev))) return rc;
  return sm_count(*dev, sms);
}

// Rows [B, L] of `width` elements of `size` bytes.
struct Span {
  const char* p;
  long long sb, sl;   // bytes
  int B, L;
  long long width;    // bytes
  const char* end() const { return p + (B - 1) * sb + (L - 1) * sl + width; }
};

Span span(const void* p, size_t size, long long sb, long long sl, int B, int L, long long width) {
  const long long s = static_cast<long long>(size);
  return Span{static_cast<const char*>(p), B > 1 ? sb * s : 0, L > 1 ? sl * s : 0, B, L, width * s};
}

// Whether two sets of rows share a byte.  Rows of equal pitch whose columns
// lie side by side do not (two slices of one buffer); any other two whose
// address ranges meet are taken to.
bool overlap(const Span& a, const Span& b) {
  if (a.end() <= b.p || b.end() <= a.p) return false;
  if (a.sl == b.sl && a.sb == b.sb && a.L > 1) {
    const long long d = ((b.p - a.p) % a.sl + a.sl) % a.sl;
    if (a.sb % a.sl == 0 && d >= a.width && d + b.width <= a.sl) return false;
  }
  return true;
}

// Rows that are written: distinct rows may not share elements.
bool rows_distinct(const Span& s) {
  if (s.L > 1 && s.sl < s.width) return s.B > 1 && s.sb >= s.width && s.sl >= (s.B - 1) * s.sb + s.width;
  return s.B <= 1 || s.sb >= (s.L - 1) * s.sl + s.width ||
         (s.sb >= s.width && s.sl >= (s.B - 1) * s.sb + s.width);
}

bool aligned(size_t to, const void* p, size_t size, std::initializer_list<long long> strides) {
  if (reinterpret_cast<uintptr_t>(p) % to) return false;
  for (long long s : strides)
    if (s * static_cast<long long>(size) % static_cast<long long>(to)) return false;
  return true;
}
bool vec16(const void* p, size_t size, std::initializer_list<long long> strides) { return aligned(16, p, size, strides); }
// Eight elements at a time: 16 bytes, or 32 of fp32.
bool vec8(const void* p, size_t size, std::initializer_list<long long> strides) { return aligned(8 * size, p, size, strides); }

int check_rows(const sol_attn_rows& r, const char* name, int B, int L) {
  if (!dtype_ok(r.dtype)) return fail(SOL_ATTN_ERR_ARG, "%s: unknown dtype %d", name, r.dtype);
  if (reinterpret_cast<uintptr_t>(r.data) % dtype_size(r.dtype))
    return fail(SOL_ATTN_ERR_ALIGN, "%s is not aligned to its elements", name);
  if ((B > 1 && r.stride_b < 0) || (L > 1 && r.stride_l < 0))
    return fail(SOL_ATTN_ERR_ARG, "%s has a negative stride", name);
  return SOL_ATTN_OK;
}

int convert(const sol_attn_vectors& v, const char* name, int B, int L, Vectors* out, bool* vec) {
  *out = Vectors{};
  if (!v.data) return SOL_ATTN_OK;
  if (!dtype_ok(v.dtype)) return fail(SOL_ATTN_ERR_ARG, "%s: unknown dtype %d", name, v.dtype);
  if (v.groups < 1 || L % v.groups)
    return fail(SOL_ATTN_ERR_ARG, "%s: %d groups do not divide %d tokens", name, v.groups, L);
  const size_t size = dtype_size(v.dtype);
  if (reinterpret_cast<uintptr_t>(v.data) % size)
    return fail(SOL_ATTN_ERR_ALIGN, "%s is not aligned to its elements", name);
  out->p = v.data;
  out->dtype = v.dtype;
  out->sb = B > 1 ? v.stride_b : 0;
  out->sg = v.groups > 1 ? v.stride_g : 0;
  out->per = L / v.groups;
  *vec = *vec && vec16(v.data, size, {out->sb, out->sg});
  return SOL_ATTN_OK;
}

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
    if (rows >= kNormRingLeast * static_cast<long long>(sms) && p.group >= kNormRingLeast && p.warps <= 8 &&
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
int launch_rope(const RopeParams& p, int dev, int sms, cudaStream_t st) {
  return p.half ? launch_rope_warps<T, true>(p, dev, sms, st) : launch_rope_warps<T, false>(p, dev, sms, st);
}

// 2-D map of rows of K elements (pitch in bytes) with a {box_k, box_rows} box
// and 128-byte swizzle; what lies outside reads as zero and is not written.
int make_map_2d(CUtensorMap* m, CUtensorMapDataType type, const void* ptr, long long K, long long rows,
                long long pitch, int box_k, int box_rows) {
  EncodeTiledFn enc;
  int rc = get_encoder(&enc);
  if (rc) return rc;
  cuuint64_t gdim[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  cuuint64_t gstride[1] = {static_cast<cuuint64_t>(pitch)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_k), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(m, type, 2, const_cast<void*>(ptr), gdim, gstride, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(SOL_ATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return SOL_ATTN_OK;
}

template <typename T>
constexpr CUtensorMapDataType map_type() {
  return sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
         : std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

struct LinearOperands {
  const int8_t* a;
  long long a_pitch;
  const int8_t* w;
  long long w_pitch;
};

template <int CG, int BN, typename T>
int launch_linear(const LinearParams& p0, const LinearOperands& o, int dev, int sms, cudaStream_t st) {
  using C = LinearConfig<CG, BN>;
  LinearParams p = p0;
  p.tiles_m = (p.M + 128 * CG - 1) / (128 * CG);
  p.tiles_n = (p.N + BN - 1) / BN;
  p.band = 8;
  const long long tiles = static_cast<long long>(p.tiles_m) * p.tiles_n;
  if (tiles > INT_MAX / 2) return fail(SOL_ATTN_ERR_UNSUPPORTED, "%lld output tiles", tiles);
  CUtensorMap ma, mw, mo{};
  int rc;
  if ((rc = make_map_2d(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, o.a, p.K, p.M, o.a_pitch, 128, 128))) return rc;
  if ((rc = make_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, o.w, p.K, p.N, o.w_pitch, 128, BN / CG))) return rc;
  p.direct = reinterpret_cast<uintptr_t>(p.out) % 16 != 0 || p.out_pitch * sizeof(T) % 16 != 0;
  if (!p.direct &&
      (rc = make_map_2d(&mo, map_type<T>(), p.out, p.N, p.M, p.out_pitch * sizeof(T), 128 / sizeof(T), 32)))
    return rc;
  static bool attr_set[kMaxDevices] = {false};   // the attribute is set per device
  if (!attr_set[dev]) {
    CUDA_TRY(cudaFuncSetAttribute(linear_kernel<CG, BN, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  static_cast<int>(C::kSmem)));
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(CG * static_cast<unsigned>(std::min<long long>(tiles, sms / CG)));
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CG;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  CUDA_TRY(cudaLaunchKernelEx(&cfg, linear_kernel<CG, BN, T>, ma, mw, mo, p));
  return SOL_ATTN_OK;
}

template <int MT, typename T>
int launch_linear_vec(const LinearParams& p, const LinearOperands& o, int sms, cudaStream_t st) {
  LinearVecParams v{p, o.a, o.a_pitch, o.w, o.w_pitch, 1};
  const int groups = (p.N + kVecRows - 1) / kVecRows;
  if (groups < kVecWarps * 8 * sms) v.split = kVecWarps;
  const int per_block = kVecWarps / v.split;
  linear_vec_kernel<MT, T><<<(groups + per_block - 1) / per_block, kVecWarps * 32, 0, st>>>(v);
  CUDA_TRY(cudaGetLastError());
  return SOL_ATTN_OK;
}

template <int BT, typename T>
int launch_linear_few(LinearParams p, const LinearOperands& o, int dev, int sms, cudaStream_t st) {
  using C = FewConfig<BT>;
  p.tiles_m = (p.M + BT - 1) / BT;
  CUtensorMap ma, mw;
  int rc;
  if ((rc = make_map_2d(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, o.a, p.K, p.M, o.a_pitch, 128, BT))) return rc;
  if ((rc = make_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, o.w, p.K, p.N, o.w_pitch, 128, 128))) return rc;
  static bool attr_set[kMaxDevices] = {false};   // the attribute is set per device
  if (!attr_set[dev]) {
    CUDA_TRY(cudaFuncSetAttribute(linear_few_kernel<BT, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  static_cast<int>(C::kSmem)));
    attr_set[dev] = true;
  }
  const int tiles = (p.N + 127) / 128 * p.tiles_m, kblocks = (p.K + 127) / 128;
  int log_split = 0;
  while (log_split < 3 && (tiles << log_split) < sms && (2 << log_split) <= kblocks) ++log_split;
  const int split = 1 << log_split;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(tiles * split);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = split;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  CUDA_TRY(cudaLaunchKernelEx(&cfg, linear_few_kernel<BT, T>, ma, mw, p, log_split));
  return SOL_ATTN_OK;
}

template <typename T>
int run_linear(const LinearParams& p, const LinearOperands& o, int dev, int sms, cudaStream_t st) {
  if (p.M == 1) return launch_linear_vec<1, T>(p, o, sms, st);
  if (p.M == 2) return launch_linear_vec<2, T>(p, o, sms, st);
  if (p.M <= 4) return launch_linear_vec<4, T>(p, o, sms, st);
  if (p.M <= 16) return launch_linear_few<16, T>(p, o, dev, sms, st);
  if (p.M <= 32) return launch_linear_few<32, T>(p, o, dev, sms, st);
  if (p.M <= kFewTokens) return launch_linear_few<64, T>(p, o, dev, sms, st);
  // The variant whose slowest SM is done first: waves of tiles, each the time
  // of its K and of its output.  A block of 128 of K takes both variants the
  // same 0.35 us, in which an SM is brought its 32 KB; the pair's tile is twice
  // as wide.  5120 channels of 5120 (us, pair / single): 200 tokens 17.9 / 16.9,
  // 512 18.6 / 28.6, 1024 32 / 41; 1034 x 1543 x 1000 14.6 / 10.0.
  const auto cost = [&](int cg, int bn) {
    const long long tiles = ((p.M + 128LL * cg - 1) / (128 * cg)) * ((p.N + bn - 1LL) / bn);
    const long long waves = (tiles + sms / cg - 1) / (sms / cg);
    return waves * ((p.K + 127) / 128 + bn / 64);
  };
  if (cost(2, 256) <= cost(1, 128)) return launch_linear<2, 256, T>(p, o, dev, sms, st);
  return launch_linear<1, 128, T>(p, o, dev, sms, st);
}

}  // namespace

extern "C" {

int sol_attn_norm_modulate(const sol_attn_norm_args* a, void* stream) {
  if (!a) return fail(SOL_ATTN_ERR_ARG, "args is NULL");
  const int B = a->B, L = a->L, C = a->C;
  int rc;
  if (B < 0 || L < 0 || C < 1) return fail(SOL_ATTN_ERR_ARG, "bad sizes B = %d, L = %d, C = %d", B, L, C);
  if (C > kMaxC) return fail(SOL_ATTN_ERR_UNSUPPORTED, "C = %d exceeds the supported maximum %d", C, kMaxC);
  if (a->norm < 0 || a->norm > 2 || a->post_norm < 0 || a->post_norm > 2)
    return fail(SOL_ATTN_ERR_ARG, "unknown norm %d or %d", a->norm, a->post_norm);
  if (!(a->eps >= 0.f) || !(a->post_eps >= 0.f)) return fail(SOL_ATTN_ERR_ARG, "eps must not be negative or NaN");
  if (B == 0 || L == 0) return SOL_ATTN_OK;
  if (static_cast<long long>(B) * L > INT_MAX) return fail(SOL_ATTN_ERR_UNSUPPORTED, "B*L exceeds 2^31 - 1");
  if (!a->x.data) return fail(SOL_ATTN_ERR_ARG, "x is NULL");
  if (!a->h.data && !a->q && !(a->x_out.data && a->y.data))
    return fail(SOL_ATTN_ERR_ARG, "no output is asked for (x_out needs y)");
  if (a->x_out.data && !a->y.data) return fail(SOL_ATTN_ERR_ARG, "x_out needs y");
  if (a->x_inner < 1 || C % a->x_inner) return fail(SOL_ATTN_ERR_ARG, "x_inner %d does not divide C", a->x_inner);
  if ((a->q == nullptr) != (a->q_scale == nullptr)) return fail(SOL_ATTN_ERR_ARG, "q and q_scale come together");

  NormParams p{};
  p.B = B, p.L = L, p.C = C;
  if ((rc = check_rows(a->x, "x", B, L))) return rc;
  const size_t xs = dtype_size(a->x.dtype);
  int ydt = a->x.dtype;   // type of y and h
  if (a->y.data) {
    if ((rc = check_rows(a->y, "y", B, L))) return rc;
    ydt = a->y.dtype;
    if (a->h.data && a->h.dtype != ydt) return fail(SOL_ATTN_ERR_UNSUPPORTED, "h must have the type of y");
  } else if (a->h.data) {
    ydt = a->h.dtype;
  }
  if (ydt != a->x.dtype && a->x.dtype != SOL_ATTN_FP32)
    return fail(SOL_ATTN_ERR_UNSUPPORTED, "y and h must have the type of x, or x must be fp32");
  const size_t ys = dtype_size(ydt);
  p.x = a->x.data;
  p.x_sb = B > 1 ? a->x.stride_b : 0, p.x_sl = L > 1 ? a->x.stride_l : 0;
  p.x_inner = a->x_inner, p.x_sh = a->x_inner < C ? a->x_stride_h : 0;
  if (p.x_sh < 0) return fail(SOL_ATTN_ERR_ARG, "x has a negative stride");
  bool vec = C % 8 == 0 && p.x_inner % 8 == 0 && vec8(p.x, xs, {p.x_sb, p.x_sl, p.x_sh});
  const Span x = span(p.x, xs, p.x_sb, p.x_sl, B, L, (C / p.x_inner - 1) * p.x_sh + p.x_inner);
  Span y{}, outs[3];
  int nouts = 0;
  if (a->y.data) {
    p.y = a->y.data, p.y_sb = B > 1 ? a->y.stride_b : 0, p.y_sl = L > 1 ? a->y.stride_l : 0;
    vec = vec && vec8(p.y, ys, {p.y_sb, p.y_sl});
    y = span(p.y, ys, p.y_sb, p.y_sl, B, L, C);
  }
  if (a->x_out.data) {
    if ((rc = check_rows(a->x_out, "x_out", B, L))) return rc;
    if (a->x_out.dtype != a->x.dtype) return fail(SOL_ATTN_ERR_UNSUPPORTED, "x_out must have the type of x");
    p.xo = a->x_out.data, p.xo_sb = B > 1 ? a->x_out.stride_b : 0, p.xo_sl = L > 1 ? a->x_out.stride_l : 0;
    vec = vec && vec8(p.xo, xs, {p.xo_sb, p.xo_sl});
    const Span s = span(p.xo, xs, p.xo_sb, p.xo_sl, B, L, C);
    // in place: each row is read whole before it is written, by the same team
    const bool in_place = p.xo == p.x && p.xo_sb == p.x_sb && p.xo_sl == p.x_sl && p.x_inner == C;
    if (!rows_distinct(s)) return fail(SOL_ATTN_ERR_ARG, "rows of x_out share elements");
    if ((!in_place && overlap(s, x)) || overlap(s, y))
      return fail(SOL_ATTN_ERR_ARG, "x_out overlaps an input (only x_out = x is allowed)");
    outs[nouts++] = s;
  }
  if (a->h.data) {
    if ((rc = check_rows(a->h, "h", B, L))) return rc;
    p.h = a->h.data, p.h_sb = B > 1 ? a->h.stride_b : 0, p.h_sl = L > 1 ? a->h.stride_l : 0;
    vec = vec && vec8(p.h, ys, {p.h_sb, p.h_sl});
    outs[nouts++] = span(p.h, ys, p.h_sb, p.h_sl, B, L, C);
    if (!rows_distinct(outs[nouts - 1])) return fail(SOL_ATTN_ERR_ARG, "rows of h share elements");
    if (overlap(outs[nouts - 1], x) || (p.y && overlap(outs[nouts - 1], y)))
      return fail(SOL_ATTN_ERR_ARG, "h overlaps an input");
  }
  if (a->q) {
    if (a->q_stride < C) return fail(SOL_ATTN_ERR_ARG, "q_stride %lld is below C", a->q_stride);
    if (reinterpret_cast<uintptr_t>(a->q_scale) % 4) return fail(SOL_ATTN_ERR_ALIGN, "q_scale is misaligned");
    p.q = a->q, p.q_sl = a->q_stride, p.q_scale = a->q_scale;
    vec = vec && reinterpret_cast<uintptr_t>(p.q) % 8 == 0 && p.q_sl % 8 == 0;
    outs[nouts++] = span(p.q, 1, p.q_sl * L, p.q_sl, B, L, C);
    if (overlap(outs[nouts - 1], x) || (p.y && overlap(outs[nouts - 1], y)))
      return fail(SOL_ATTN_ERR_ARG, "q overlaps an input");
  }
  for (int i = 0; i < nouts; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return fail(SOL_ATTN_ERR_ARG, "two outputs overlap");
  if ((rc = convert(a->scale, "scale", B, L, &p.scale, &vec)) || (rc = convert(a->shift, "shift", B, L, &p.shift, &vec)) ||
      (rc = convert(a->gate, "gate", B, L, &p.gate, &vec)) || (rc = convert(a->weight, "weight", B, L, &p.weight, &vec)) ||
      (rc = convert(a->bias, "bias", B, L, &p.bias, &vec)) ||
      (rc = convert(a->post_weight, "post_weight", B, L, &p.post_weight, &vec)) ||
      (rc = convert(a->post_bias, "post_bias", B, L, &p.post_bias, &vec)))
    return rc;
  const sol_attn_vectors* vectors[7] = {&a->scale, &a->shift, &a->gate, &a->weight, &a->bias, &a->post_weight, &a->post_bias};
  for (const sol_attn_vectors* v : vectors) {
    if (!v->data) continue;
    const Span s = span(v->data, dtype_size(v->dtype), v->stride_b, v->stride_g, B, v->groups, C);
    for (int i = 0; i < nouts; ++i)
      if (overlap(outs[i], s)) return fail(SOL_ATTN_ERR_ARG, "an output overlaps a vector of parameters");
  }
  p.group = L;
  for (const Vectors* v : {&p.scale, &p.shift, &p.gate})
    if (v->p) p.group = std::gcd(p.group, v->per);
  p.channels = static_cast<float>(C), p.inv_channels = 1.f / p.channels;
  p.rs = a->residual_scale;
  p.pre = a->norm, p.post = a->post_norm;
  p.pre_eps = a->eps, p.post_eps = a->post_eps;

  // whether 32-byte vectors can read and write the rows of a 16-bit type
  const bool wide = p.x_inner % 16 == 0 && aligned(32, p.x, xs, {p.x_sb, p.x_sl, p.x_sh}) && aligned(32, p.y, ys, {p.y_sb, p.y_sl}) &&
                    aligned(32, p.xo, xs, {p.xo_sb, p.xo_sl}) && aligned(32, p.h, ys, {p.h_sb, p.h_sl}) &&
                    aligned(16, p.q, 1, {p.q_sl});
  int dev, sms;
  if ((rc = device(&dev, &sms))) return rc;
  auto st = static_cast<cudaStream_t>(stream);
  if (a->x.dtype == SOL_ATTN_BF16) return launch_norm_res<__nv_bfloat16, __nv_bfloat16>(p, vec, wide, dev, sms, st);
  if (a->x.dtype == SOL_ATTN_FP16) return launch_norm_res<__half, __half>(p, vec, wide, dev, sms, st);
  if (ydt == SOL_ATTN_BF16) return launch_norm_res<float, __nv_bfloat16>(p, vec, wide, dev, sms, st);
  if (ydt == SOL_ATTN_FP16) return launch_norm_res<float, __half>(p, vec, wide, dev, sms, st);
  return launch_norm_res<float, float>(p, vec, wide, dev, sms, st);
}

int sol_attn_rope(const sol_attn_rope_args* a, void* stream) {
  if (!a) return fail(SOL_ATTN_ERR_ARG, "args is NULL");
  const int B = a->B, L = a->L, H = a->H, d = a->d;
  int rc;
  if (B < 0 || L < 0 || H < 1 || d < 1) return fail(SOL_ATTN_ERR_ARG, "bad sizes B = %d, L = %d, H = %d, d = %d", B, L, H, d);
  if (d % 16 || d > kRopeMaxD) return fail(SOL_ATTN_ERR_UNSUPPORTED, "d must be a multiple of 16 up to 256 (got %d)", d);
  if (static_cast<long long>(H) * d > kMaxC)
    return fail(SOL_ATTN_ERR_UNSUPPORTED, "H*d = %lld exceeds the supported maximum %d", static_cast<long long>(H) * d, kMaxC);
  if (!dtype_ok(a->dtype)) return fail(SOL_ATTN_ERR_ARG, "unknown dtype %d", a->dtype);
  if (a->norm < 0 || a->norm > 2) return fail(SOL_ATTN_ERR_ARG, "unknown norm %d", a->norm);
  if (!(a->eps >= 0.f)) return fail(SOL_ATTN_ERR_ARG, "eps must not be negative or NaN");
  if (a->pairing != SOL_ATTN_PAIR_INTERLEAVED && a->pairing != SOL_ATTN_PAIR_HALF)
    return fail(SOL_ATTN_ERR_ARG, "unknown pairing %d", a->pairing);
  if (!a->freqs || !a->axis) return fail(SOL_ATTN_ERR_ARG, "freqs or axis is NULL");
  if (a->axes < 1 || a->axes > kRopeMaxAxes) return fail(SOL_ATTN_ERR_UNSUPPORTED, "%d axes (1 to %d)", a->axes, kRopeMaxAxes);
  RopeParams p{};
  for (int i = 0; i < d / 2; ++i) {
    if (!std::isfinite(a->freqs[i])) return fail(SOL_ATTN_ERR_ARG, "frequency %d is not finite", i);
    if (a->axis[i] >= a->axes) return fail(SOL_ATTN_ERR_ARG, "pair %d is on axis %d of %d", i, a->axis[i], a->axes);
    p.turns[i] = a->freqs[i] / 6.283185307179586476925286766559;
    p.axis[i] = a->axis[i];
  }
  if (a->pos_kind == SOL_ATTN_POS_GRID) {
    const long long f = a->grid_f, h = a->grid_h, w = a->grid_w;
    if (a->axes != 3) return fail(SOL_ATTN_ERR_ARG, "a grid has 3 axes");
    if (f < 1 || h < 1 || w < 1 || f > INT_MAX / h || f * h > INT_MAX / w)
      return fail(SOL_ATTN_ERR_ARG, "bad grid %lld x %lld x %lld", f, h, w);
    if (a->start < 0) return fail(SOL_ATTN_ERR_ARG, "start is negative");
    p.grid_h = a->grid_h, p.grid_w = a->grid_w, p.grid_tokens = f * h * w, p.start = a->start;
  } else {
    if (a->pos_kind < SOL_ATTN_POS_GRID || a->pos_kind > SOL_ATTN_POS_F64)
      return fail(SOL_ATTN_ERR_ARG, "unknown kind of positions %d", a->pos_kind);
    p.pos = a->positions;
    p.pos_sb = B > 1 ? a->pos_stride_b : 0, p.pos_sl = L > 1 ? a->pos_stride_l : 0, p.pos_sa = a->axes > 1 ? a->pos_stride_a : 0;
    if (p.pos_sb < 0 || p.pos_sl < 0 || p.pos_sa < 0) return fail(SOL_ATTN_ERR_ARG, "positions has a negative stride");
  }
  p.pos_kind = a->pos_kind;
  if (B == 0 || L == 0) return SOL_ATTN_OK;
  if (static_cast<long long>(B) * L > INT_MAX) return fail(SOL_ATTN_ERR_UNSUPPORTED, "B*L exceeds 2^31 - 1");
  if (p.pos_kind != kPosGrid) {
    const size_t s = p.pos_kind == kPosI32 || p.pos_kind == kPosF32 ? 4 : 8;
    if (!p.pos) return fail(SOL_ATTN_ERR_ARG, "positions is NULL");
    if (reinterpret_cast<uintptr_t>(p.pos) % s) return fail(SOL_ATTN_ERR_ALIGN, "positions is not aligned to its elements");
  }
  p.B = B, p.L = L, p.H = H, p.d = d;
  p.norm = a->norm, p.eps = a->eps;
  p.inv_channels = 1.f / static_cast<float>(p.norm == kRopeNormToken ? H * d : d);
  p.half = a->pairing == SOL_ATTN_PAIR_HALF;
  const size_t size = dtype_size(a->dtype);
  const long long n = static_cast<long long>(B) * H * L * d;
  const sol_attn_rope_tensor* in[3] = {&a->q, &a->k, &a->v};
  RopeTensor* out[3] = {&p.q, &p.k, &p.v};
  const char* names[3] = {"q", "k", "v"};
  for (int i = 0; i < 3; ++i) {
    const sol_attn_rope_tensor& t = *in[i];
    if (i == 2 && !t.in && !t.out) continue;
    if ((rc = check_ptr(t.in, names[i])) || (rc = check_ptr(t.out, names[i]))) return rc;
    RopeTensor& r = *out[i];
    r.in = t.in, r.out = t.out;
    r.sb = B > 1 ? t.stride_b : 0, r.sl = L > 1 ? t.stride_l : 0, r.sh = H > 1 ? t.stride_h : 0;
    if (r.sb < 0 || r.sl < 0 || r.sh < 0) return fail(SOL_ATTN_ERR_ARG, "%s has a negative stride", names[i]);
    if (!vec8(t.in, size, {r.sb, r.sl, r.sh}) || !vec8(t.out, size, {}))
      return fail(SOL_ATTN_ERR_ALIGN, "%s: base and strides must be multiples of 8 elements", names[i]);
    if (i < 2 && t.weight) {
      if (a->norm == kRopeNormNone) return fail(SOL_ATTN_ERR_ARG, "%s has a weight but no norm", names[i]);
      if (!dtype_ok(t.weight_dtype)) return fail(SOL_ATTN_ERR_ARG, "%s weight: unknown dtype %d", names[i], t.weight_dtype);
      if (reinterpret_cast<uintptr_t>(t.weight) % 16) return fail(SOL_ATTN_ERR_ALIGN, "%s weight is not 16-byte aligned", names[i]);
      r.weight = t.weight, r.weight_dtype = t.weight_dtype;
    }
  }
  const int tensors = p.v.in ? 3 : 2;
  p.packed = 1;
  for (int i = 0; i < tensors; ++i) p.packed = p.packed && (out[i]->sh == d || H == 1);
  // a head's place in the output is kept in 32 bits, by 8 elements
  if (static_cast<long long>(H) * d / 8 * L > UINT_MAX)
    return fail(SOL_ATTN_ERR_UNSUPPORTED, "H*L*d = %lld exceeds 2^35", static_cast<long long>(H) * d * L);
  for (int i = 0; i < tensors; ++i) {
    const char* o = static_cast<const char*>(out[i]->out);
    const char* o_end = o + n * static_cast<long long>(size);
    for (int j = 0; j < tensors; ++j) {
      const RopeTensor& t = *out[j];
      const char* x = static_cast<const char*>(t.in);
      const char* x_end = x + ((B - 1) * t.sb + (L - 1) * t.sl + (H - 1) * t.sh + d) * static_cast<long long>(size);
      if (o < x_end && x < o_end) return fail(SOL_ATTN_ERR_ARG, "an output overlaps an input tensor");
      const char* o2 = static_cast<const char*>(t.out);
      if (j != i && o < o2 + n * static_cast<long long>(size) && o2 < o_end)
        return fail(SOL_ATTN_ERR_ARG, "two outputs overlap");
    }
  }
  for (int i = 0; i < tensors; ++i) {
    const Span o = span(out[i]->out, size, 0, 0, 1, 1, n);
    for (int j = 0; j < 2; ++j)
      if (out[j]->weight &&
          overlap(o, span(out[j]->weight, dtype_size(out[j]->weight_dtype), 0, 0, 1, 1, p.norm == kRopeNormToken ? H * d : d)))
        return fail(SOL_ATTN_ERR_ARG, "an output overlaps a weight");
    if (p.pos && overlap(o, span(p.pos, p.pos_kind == kPosI32 || p.pos_kind == kPosF32 ? 4 : 8, 0, 0, 1, 1,
                                 (B - 1) * p.pos_sb + (L - 1) * p.pos_sl + (a->axes - 1) * p.pos_sa + 1)))
      return fail(SOL_ATTN_ERR_ARG, "an output overlaps the positions");
  }
  int dev, sms;
  if ((rc = device(&dev, &sms))) return rc;
  auto st = static_cast<cudaStream_t>(stream);
  if (a->dtype == SOL_ATTN_BF16) return launch_rope<__nv_bfloat16>(p, dev, sms, st);
  if (a->dtype == SOL_ATTN_FP16) return launch_rope<__half>(p, dev, sms, st);
  return launch_rope<float>(p, dev, sms, st);
}

int sol_attn_quantized_linear(const sol_attn_linear_args* a, void* stream) {
  if (!a) return fail(SOL_ATTN_ERR_ARG, "args is NULL");
  const int M = a->M, N = a->N, K = a->K;
  int rc;
  if (M < 0 || N < 0 || K < 1) return fail(SOL_ATTN_ERR_ARG, "bad sizes M = %d, N = %d, K = %d", M, N, K);
  if (M > INT_MAX - 512 || N > INT_MAX - 512) return fail(SOL_ATTN_ERR_UNSUPPORTED, "M = %d or N = %d is too large", M, N);
  if (a->flags & ~SOL_ATTN_FLAG_TEST_STALL) return fail(SOL_ATTN_ERR_ARG, "unknown flag bits 0x%x", a->flags);
  if (K > kMaxLinearK) return fail(SOL_ATTN_ERR_UNSUPPORTED, "K = %d exceeds %d, up to which the sums fit 32 bits", K, kMaxLinearK);
  if (!dtype_ok(a->out_dtype)) return fail(SOL_ATTN_ERR_ARG, "out: unknown dtype %d", a->out_dtype);
  if (M == 0 || N == 0) return SOL_ATTN_OK;
  if ((rc = check_ptr(a->a, "a")) || (rc = check_ptr(a->w, "w"))) return rc;
  if (!a->a_scale || !a->w_scale || !a->out) return fail(SOL_ATTN_ERR_ARG, "a_scale, w_scale or out is NULL");
  if ((M > 1 && a->a_stride < K) || (N > 1 && a->w_stride < K))
    return fail(SOL_ATTN_ERR_ARG, "a row pitch is below K");
  if ((M > 1 && a->a_stride % 16) || (N > 1 && a->w_stride % 16))
    return fail(SOL_ATTN_ERR_ALIGN, "the rows of a and w must start at multiples of 16 bytes");
  if (M > 1 && a->out_stride < N) return fail(SOL_ATTN_ERR_ARG, "out_stride is below N");
  const size_t size = dtype_size(a->out_dtype);
  if (reinterpret_cast<uintptr_t>(a->a_scale) % 4 || reinterpret_cast<uintptr_t>(a->w_scale) % 4 ||
      reinterpret_cast<uintptr_t>(a->out) % size)
    return fail(SOL_ATTN_ERR_ALIGN, "a_scale, w_scale or out is not aligned to its elements");
  LinearParams p{};
  p.M = M, p.N = N, p.K = K;
  p.a_scale = a->a_scale, p.w_scale = a->w_scale;
  p.stall = (a->flags & SOL_ATTN_FLAG_TEST_STALL) != 0;
  p.timeout_ns = p.stall ? 1000000ull : 2000000000ull;
  if (a->bias) {
    if (!dtype_ok(a->bias_dtype)) return fail(SOL_ATTN_ERR_ARG, "bias: unknown dtype %d", a->bias_dtype);
    if (reinterpret_cast<uintptr_t>(a->bias) % dtype_size(a->bias_dtype))
      return fail(SOL_ATTN_ERR_ALIGN, "bias is not aligned to its elements");
    p.bias = a->bias, p.bias_dtype = a->bias_dtype;
  }
  // a pitch that no row uses may be anything: the maps take one that fits
  const long long fit = (K + 15LL) / 16 * 16;
  LinearOperands o{a->a, M > 1 ? a->a_stride : fit, a->w, N > 1 ? a->w_stride : fit};
  p.out = a->out;
  p.out_pitch = M > 1 ? a->out_stride : (N + 7LL) / 8 * 8;
  const Span out = span(p.out, size, 0, p.out_pitch, 1, M, N);
  if (overlap(out, span(o.a, 1, 0, o.a_pitch, 1, M, K)) || overlap(out, span(o.w, 1, 0, o.w_pitch, 1, N, K)) ||
      overlap(out, span(p.a_scale, 4, 0, 0, 1, 1, M)) || overlap(out, span(p.w_scale, 4, 0, 0, 1, 1, N)) ||
      (p.bias && overlap(out, span(p.bias, dtype_size(p.bias_dtype), 0, 0, 1, 1, N))))
    return fail(SOL_ATTN_ERR_ARG, "out overlaps an input");
  int dev, sms;
  if ((rc = device(&dev, &sms))) return rc;
  auto st = static_cast<cudaStream_t>(stream);
  if (a->out_dtype == SOL_ATTN_BF16) return run_linear<__nv_bfloat16>(p, o, dev, sms, st);
  if (a->out_dtype == SOL_ATTN_FP16) return run_linear<__half>(p, o, dev, sms, st);
  return run_linear<float>(p, o, dev, sms, st);
}

int sol_attn_linear_status(void* stream) {
  int dev, sms, rc;
  if ((rc = device(&dev, &sms))) return rc;
  auto st = static_cast<cudaStream_t>(stream);
  CUDA_TRY(cudaStreamSynchronize(st));
  unsigned h = 0;
  CUDA_TRY(cudaMemcpyFromSymbol(&h, g_linear_status, sizeof(h)));
  if (!h) return SOL_ATTN_OK;
  const unsigned zero = 0;
  CUDA_TRY(cudaMemcpyToSymbol(g_linear_status, &zero, sizeof(zero)));
  if (h & 1u) return fail(SOL_ATTN_ERR_TIMEOUT, "a bounded device wait of a product gave up (status 0x%x)", h);
  return fail(SOL_ATTN_ERR_DEVICE, "a product's shared memory is not aligned to its tiles (status 0x%x)", h);
}

}  // extern "C"
