// linear_launch.cu — launches of the kernels for products of 8-bit integers.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "host.h"
#include "layer_launch.h"

namespace solattn {
namespace {

// Tokens up to which channels are the rows of the tile (15360 x 5120: 128 tokens
// in tiles of 64 23 us, in one tile of 128 rows 37; 5120 x 5120: 200 tokens 19
// against 16.6 the other way round).
constexpr int kFewTokens = 128;

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

template <int CG, int BN, typename T>
int launch_linear_tiles(const LinearParams& p0, const LinearOperands& o, int dev, int sms, cudaStream_t st) {
  using C = LinearConfig<CG, BN>;
  LinearParams p = p0;
  p.tiles_m = (p.M + 128 * CG - 1) / (128 * CG);
  p.tiles_n = (p.N + BN - 1) / BN;
  // Tiles of M that share each tile of the weights while it lies in L2.  Weights
  // that stay there whole, a quarter of its 126 MB or less, want narrow bands, whose
  // tokens are read once; larger ones pass through L2 once a band.  us with
  // 2, 4, 8, 16, 32 (rows x channels x K, MB of weights):
  //   16  32768 x  2048 x  8192   340   340   342   352   380
  //   18  32768 x  9216 x  2048   417   418   423   425   422
  //   25  75600 x  5120 x  5120  1207  1213  1222  1236  1243
  //   64   8192 x  8192 x  8192   374   356   345   336   366
  //   67  75600 x  5120 x 13824  3554  3587  3419  3447  3711
  //   75  75600 x 15360 x  5120  4015  4004  3783  3672  3697
  //  144   4096 x 24576 x  6144   443   409   390   377   377
  p.band = static_cast<long long>(p.N) * p.K <= (32 << 20) ? 2 : 16;
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

__global__ void take_linear_status(unsigned* taken) { *taken = atomicExch(&g_linear_status, 0u); }

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
  if (cost(2, 256) <= cost(1, 128)) return launch_linear_tiles<2, 256, T>(p, o, dev, sms, st);
  return launch_linear_tiles<1, 128, T>(p, o, dev, sms, st);
}

}  // namespace

int launch_linear(const LinearParams& p, const LinearOperands& o, int dtype, int dev, int sms, cudaStream_t st) {
  if (dtype == SOL_ATTN_BF16) return run_linear<__nv_bfloat16>(p, o, dev, sms, st);
  if (dtype == SOL_ATTN_FP16) return run_linear<__half>(p, o, dev, sms, st);
  return run_linear<float>(p, o, dev, sms, st);
}

int read_linear_status(cudaStream_t st, unsigned* status) {
  // Taken in one step behind the stream's products, so that what another
  // stream's product reports meanwhile is left for the next reading, and with
  // nothing on the default stream, which would wait for unrelated work.
  cudaStreamCaptureStatus capture;
  CUDA_TRY(cudaStreamIsCapturing(st, &capture));
  if (capture != cudaStreamCaptureStatusNone) return fail(SOL_ATTN_ERR_STATE, "the stream is being captured: it cannot be synchronised");
  unsigned* taken = nullptr;
  CUDA_TRY(cudaMallocAsync(&taken, sizeof(*taken), st));
  take_linear_status<<<1, 1, 0, st>>>(taken);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaMemcpyAsync(status, taken, sizeof(*taken), cudaMemcpyDeviceToHost, st);
  const cudaError_t freed = cudaFreeAsync(taken, st), done = cudaStreamSynchronize(st);
  CUDA_TRY(e != cudaSuccess ? e : freed != cudaSuccess ? freed : done);
  return SOL_ATTN_OK;
}

}  // namespace solattn
