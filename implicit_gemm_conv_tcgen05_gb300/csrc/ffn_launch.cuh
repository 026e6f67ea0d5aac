// Launches of the feed-forward GEMM kernels: tile width, schedule, tensor maps.
#pragma once

#include <mutex>

#include "ffn_host.h"
#include "ffn_skinny.cuh"
#include "ffn_tc.cuh"
#include "launch.cuh"

namespace igc {

// Largest number of rows of X that the swapped (decode) kernel takes; above it the
// 256-row tiles are used.
constexpr int kSkinnyMaxM = 128;

struct FfnOperands {
  CUtensorMap a[2], b[2];
};

template <FfnOp kOp, int BN>
int ffn_kernel_setup(const DeviceInfo& dev, int* max_clusters) {
  static std::once_flag once[64];
  static int rc[64], clusters[64];
  const int d = dev.device;
  std::call_once(once[d], [&] {
    using Cfg = FfnCfg<kOp, BN>;
    rc[d] = IGC_ERR_CUDA;
    if (dev.smem_optin < Cfg::kSmemBytes) {
      rc[d] = IGC_ERR_UNSUPPORTED;
      return;
    }
    auto kern = igc_ffn_gemm_kernel<kOp, BN>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(Cfg::kSmemBytes)) != cudaSuccess)
      return;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (dev.sm_count / 2), 1, 1);
    cfg.blockDim = dim3(kFfnThreads, 1, 1);
    cfg.dynamicSmemBytes = Cfg::kSmemBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) {
      (void)cudaGetLastError();
      n = dev.sm_count / 2;
    }
    clusters[d] = n;
    rc[d] = n > 0 ? IGC_OK : IGC_ERR_UNSUPPORTED;
  });
  *max_clusters = clusters[d];
  return rc[d];
}

// Estimated time of the schedule at tile width bn (in units of one 256-wide tile):
// rounds over the CTA pairs, a last round of column halves counting one half, times
// the width over its relative rate (kBnEff's measurements).
inline double ffn_cost(long long tiles_m, long long N, int out_n, bool halves, double eff,
                       int clusters) {
  const long long tiles = tiles_m * ((N + out_n - 1) / out_n);
  const long long rem = tiles % clusters;
  const double rounds = static_cast<double>(tiles / clusters) +
                        (rem == 0 ? 0.0 : (halves && 2 * rem <= clusters ? 0.5 : 1.0));
  return rounds * out_n / eff;
}

template <FfnOp kOp, int BN>
int ffn_launch_bn(const DeviceInfo& dev, const FfnOperands& ops, const CUtensorMap* out_maps,
                  FfnParams p, cudaStream_t stream) {
  using Cfg = FfnCfg<kOp, BN>;
  int max_clusters = 0;
  int rc = ffn_kernel_setup<kOp, BN>(dev, &max_clusters);
  if (rc != IGC_OK) return rc;
  p.tiles_m = static_cast<int>((static_cast<long long>(p.M) + BM - 1) / BM);
  p.tiles_n = static_cast<int>((static_cast<long long>(p.N) + Cfg::kOutN - 1) / Cfg::kOutN);
  const long long tiles = static_cast<long long>(p.tiles_m) * p.srcs * p.tiles_n;
  if (tiles > 0x3fff0000LL) return IGC_ERR_UNSUPPORTED;
  p.num_tiles = static_cast<int>(tiles);
  p.group_m = p.tiles_m * p.srcs < 8 ? p.tiles_m * p.srcs : 8;
  p.tail_start = Cfg::kHalves ? tail_start_of(p.num_tiles, max_clusters) : p.num_tiles;
  p.num_units = p.num_tiles + (p.num_tiles - p.tail_start);
  p.wait_limit_ns = wait_limit_ns();
  p.status = status_word();
  const int clusters = p.num_units < max_clusters ? p.num_units : max_clusters;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * clusters, 1, 1);
  cfg.blockDim = dim3(kFfnThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, igc_ffn_gemm_kernel<kOp, BN>, ops.a[0], ops.a[1], ops.b[0],
                         ops.b[1], out_maps[0], out_maps[1], out_maps[2], p) != cudaSuccess) {
    (void)cudaGetLastError();
    return IGC_ERR_CUDA;
  }
  return IGC_OK;
}

// Fills output slot i of p and its tensor map (bulk stores where the matrix allows TMA:
// boxes of 32 rows x 128 bytes).
inline void ffn_set_out(FfnParams& p, CUtensorMap* maps, int i, const Mat& m) {
  FfnOut& o = p.out[i];
  o.ptr = const_cast<void*>(m.ptr);
  o.ld = m.ld;
  o.f32 = m.dtype == IGC_F32;
  o.vec = 0;
  o.tma = 0;
  if (m.ptr == nullptr) return;
  const size_t es = elem_size(m.dtype);
  o.vec = rows_aligned(m.ptr, m.ld, es, 16);
  if (o.vec)
    o.tma = encode_tiled_2d_fresh(&maps[i], map_type(m.dtype), m.ptr,
                                  static_cast<uint64_t>(p.N), static_cast<uint64_t>(p.M),
                                  static_cast<uint64_t>(m.ld) * es,
                                  static_cast<uint32_t>(128 / es), 32) == IGC_OK;
}

// Tensor map of a rows x cols operand: K-major boxes are 64 k x box_rows rows;
// MN-major boxes are 64 outputs x one stage of k.
inline int ffn_operand_map(CUtensorMap* map, int dtype, const Mat& m, int64_t rows, int64_t cols,
                           bool mn_major, int box_rows) {
  return encode_tiled_2d_fresh(map, map_type(dtype), m.ptr, static_cast<uint64_t>(cols),
                               static_cast<uint64_t>(rows), static_cast<uint64_t>(m.ld) * 2, BK,
                               static_cast<uint32_t>(mn_major ? kFfnKS : box_rows));
}

// Chooses the tile width, encodes the operand maps and launches.  A[i] is a_rows x
// a_cols, B[i] b_rows x b_cols; p holds M, N, kb_seg, segs, srcs and the epilogue.
template <FfnOp kOp>
int ffn_launch(const DeviceInfo& dev, int dtype, int count_a, const Mat* A, int64_t a_rows,
               int64_t a_cols, int count_b, const Mat* B, int64_t b_rows, int64_t b_cols,
               const Mat* outs, int n_outs, FfnParams p, cudaStream_t stream) {
  int clusters = 0;
  int rc = ffn_kernel_setup<kOp, 256>(dev, &clusters);
  if (rc != IGC_OK) return rc;
  p.bf16 = dtype == IGC_BF16;
  const long long tm = (static_cast<long long>(p.M) + BM - 1) / BM * p.srcs;
  const int wide = FfnCfg<kOp, 256>::kOutN, narrow = FfnCfg<kOp, 128>::kOutN;
  int bn = ffn_cost(tm, p.N, wide, true, kBnEff[0], clusters) <=
                   ffn_cost(tm, p.N, narrow, false, kBnEff[2], clusters)
               ? 256
               : 128;
  bn = tile_width_override() == 128 || tile_width_override() == 256 ? tile_width_override() : bn;
  FfnOperands ops = {};
  for (int i = 0; i < count_a; ++i) {
    rc = ffn_operand_map(&ops.a[i], dtype, A[i], a_rows, a_cols, ffn_a_mn(kOp), BM_CTA);
    if (rc != IGC_OK) return rc;
  }
  for (int i = 0; i < count_b; ++i) {
    rc = ffn_operand_map(&ops.b[i], dtype, B[i], b_rows, b_cols, ffn_b_mn(kOp), bn / 4);
    if (rc != IGC_OK) return rc;
  }
  CUtensorMap out_maps[3] = {};
  for (int i = 0; i < n_outs; ++i) ffn_set_out(p, out_maps, i, outs[i]);
  return bn == 256 ? ffn_launch_bn<kOp, 256>(dev, ops, out_maps, p, stream)
                   : ffn_launch_bn<kOp, 128>(dev, ops, out_maps, p, stream);
}

// ---------------------------------------------------------------------------
// few rows of X: the swapped kernel
// ---------------------------------------------------------------------------
constexpr size_t kSkinnySmem = 110 * 1024;  // two CTAs on an SM

template <bool kGated>
int ffn_launch_skinny(const DeviceInfo& dev, int dtype, int64_t K, const Mat& X, const Mat* W,
                      SkinnyParams p, const Mat* outs, int n_outs, cudaStream_t stream) {
  static std::once_flag once[64];
  static int rcs[64];
  auto kern = igc_ffn_skinny_kernel<kGated>;
  std::call_once(once[dev.device], [&] {
    rcs[dev.device] =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSkinnySmem)) == cudaSuccess
            ? IGC_OK
            : IGC_ERR_CUDA;
  });
  if (rcs[dev.device] != IGC_OK) return rcs[dev.device];

  const int out_t = kGated ? kSkRows / 2 : kSkRows;
  const long long blocks = (static_cast<long long>(p.N) + out_t - 1) / out_t;
  p.mt = (p.M + 15) / 16 * 16;
  p.tmem_cols = 32;
  while (p.tmem_cols < static_cast<uint32_t>(p.mt)) p.tmem_cols *= 2;
  p.atoms = static_cast<int>((K + BK - 1) / BK);
  // CTAs per block: as many as keep the grid within two CTAs per SM and leave each
  // at least four 64-k steps
  p.split = 1;
  while (p.split < kSkMaxSplit && 2 * p.split * blocks <= 2LL * dev.sm_count &&
         p.atoms >= 8 * p.split)
    p.split *= 2;
  p.per_cta = (p.atoms + p.split - 1) / p.split;
  if (blocks * p.split > 0x7fffffffLL) return IGC_ERR_UNSUPPORTED;
  const size_t stage = kSkWBytes + static_cast<size_t>(p.mt) * BK * 2;
  const size_t part = static_cast<size_t>(p.mt) * kSkRows * 4;
  size_t stages = (kSkinnySmem - 1024) / stage;
  if (stages > kSkMaxStages) stages = kSkMaxStages;
  if (stages > static_cast<size_t>(p.per_cta)) stages = static_cast<size_t>(p.per_cta);
  p.stages = static_cast<int>(stages);
  const size_t ring = stages * stage;
  p.bf16 = dtype == IGC_BF16;
  p.wait_limit_ns = wait_limit_ns();
  p.status = status_word();
  for (int i = 0; i < n_outs; ++i) {
    p.out[i] = const_cast<void*>(outs[i].ptr);
    p.ld[i] = outs[i].ld;
    p.f32[i] = outs[i].dtype == IGC_F32;
    p.vec[i] = rows_aligned(outs[i].ptr, outs[i].ld, elem_size(outs[i].dtype),
                            4 * elem_size(outs[i].dtype));
  }
  CUtensorMap mx, mw[2];
  int rc = ffn_operand_map(&mx, dtype, X, p.M, K, false, p.mt);
  if (rc != IGC_OK) return rc;
  for (int i = 0; i < 2; ++i) {
    rc = ffn_operand_map(&mw[i], dtype, W[kGated ? i : 0], p.N, K, false, out_t);
    if (rc != IGC_OK) return rc;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks * p.split), 1, 1);
  cfg.blockDim = dim3(kSkThreads, 1, 1);
  cfg.dynamicSmemBytes = 1024 + (ring > part ? ring : part);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kern, mx, mw[0], mw[1], p) != cudaSuccess) {
    (void)cudaGetLastError();
    return IGC_ERR_CUDA;
  }
  return IGC_OK;
}

}  // namespace igc
