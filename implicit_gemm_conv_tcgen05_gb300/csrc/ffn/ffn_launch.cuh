// Launches of the feed-forward GEMM kernels: tile width, schedule, tensor maps.
#pragma once

#include <algorithm>
#include <cmath>
#include <mutex>

#include "ffn_host.h"
#include "ffn_small.cuh"
#include "ffn_tc.cuh"
#include "launch.cuh"

namespace igc {

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
  o.tma = 0;
  if (m.ptr == nullptr) return;
  const size_t es = elem_size(m.dtype);
  o.whole = static_cast<size_t>(p.N) * es % 16 == 0;
  if (rows_aligned(m.ptr, m.ld, es, 16))
    o.tma = encode_tiled_2d_fresh(&maps[i], map_type(m.dtype), m.ptr,
                                  static_cast<uint64_t>(p.N), static_cast<uint64_t>(p.M),
                                  static_cast<uint64_t>(m.ld) * es,
                                  static_cast<uint32_t>(128 / es), 32) == IGC_OK;
}

// Tensor map of a rows x cols operand: K-major boxes are 64 k x box_rows rows;
// MN-major boxes are 64 outputs x box_rows k.
inline int ffn_operand_map(CUtensorMap* map, int dtype, const Mat& m, int64_t rows, int64_t cols,
                           int box_rows) {
  return encode_tiled_2d_fresh(map, map_type(dtype), m.ptr, static_cast<uint64_t>(cols),
                               static_cast<uint64_t>(rows), static_cast<uint64_t>(m.ld) * 2, BK,
                               static_cast<uint32_t>(box_rows));
}

// A product of the feed-forward operators: out[m, n] = sum over segments and k of
// A[m, k] B[n, k] (A the output's rows, B its columns; either may be stored with the
// output index contiguous, see ffn_tc.cuh), and what the epilogue takes.
struct FfnProblem {
  int64_t M = 0, N = 0, K = 0;  // one output matrix, one contraction segment
  int dtype = IGC_BF16;
  int segs = 1, srcs = 1;
  Mat A[2], B[2];               // count_a / count_b of them
  int count_a = 1, count_b = 1;
  Mat out[3];
  int act = IGC_ACT_NONE;
  const void* bias[2] = {};
  int bias_dtype = IGC_F32;
  Mat R;
  bool late_wait = false;       // see ffn_dependency_wait
};

// An operand of `cols` columns that a plan takes to start on a 16-byte boundary and to be
// closely packed.
inline Mat packed_rows(int64_t cols) {
  Mat m;
  m.ld = (cols + 7) / 8 * 8;
  return m;
}

// The products of a backward pass as they are planned: dX = sum_s D[s] W[s] and
// dW[s] = D[s]^T X over closely packed operands (D M x N, W N x K, X M x K).
inline FfnProblem grad_x_problem(int64_t M, int64_t N, int64_t K, int dtype, int count) {
  FfnProblem q;
  q.M = M, q.N = K, q.K = N, q.dtype = dtype;
  q.segs = q.count_a = q.count_b = count;
  for (int i = 0; i < count; ++i) q.A[i] = packed_rows(N), q.B[i] = packed_rows(K);
  return q;
}
inline FfnProblem grad_w_problem(int64_t M, int64_t N, int64_t K, int dtype, int count) {
  FfnProblem q;
  q.M = N, q.N = K, q.K = M, q.dtype = dtype;
  q.srcs = q.count_a = count;
  for (int i = 0; i < count; ++i) q.A[i] = packed_rows(N);
  q.B[0] = packed_rows(K);
  return q;
}

// Stored extents of operand i: MN-major operands have k as their rows.
inline int ffn_map_a(CUtensorMap* map, const FfnProblem& q, int i, bool mn, int box_rows) {
  return mn ? ffn_operand_map(map, q.dtype, q.A[i], q.K, q.M, box_rows)
            : ffn_operand_map(map, q.dtype, q.A[i], q.M, q.K, box_rows);
}
inline int ffn_map_b(CUtensorMap* map, const FfnProblem& q, int i, bool mn, int box_rows) {
  return mn ? ffn_operand_map(map, q.dtype, q.B[i], q.K, q.N, box_rows)
            : ffn_operand_map(map, q.dtype, q.B[i], q.N, q.K, box_rows);
}

// Estimated times in microseconds, for choosing between schedules (measured on GB300: a
// CTA takes in about 65 bytes a nanosecond through TMA, two on an SM 95 together, one with
// twice the stages 85; an SM reads about 40 from the shared memory of the other CTAs of
// its cluster; back-to-back calls get 4.4 TB/s from DRAM with 64 streaming CTAs each, 6.0
// with 128 and 7.3 with 256; a launch and a CTA's set-up, first loads and last stores take
// about 3.5 us, a further wave of CTAs about 4).
constexpr double kUsFixed = 3.5, kCtaRate = 65e3, kTwoCtaRate = 95e3, kDeepCtaRate = 85e3,
                 kDsmemPerSm = 40e3, kDramMost = 9.3e6, kDramRate = 6.6e6, kUsWave = 4.0;

// Bytes of the operands, each read once.
template <FfnOp kOp>
double operand_bytes(const FfnProblem& q) {
  return 2.0 * q.segs * static_cast<double>(q.K) *
         (static_cast<double>(q.N) * (kOp == FfnOp::Gated ? 2 : 1) +
          static_cast<double>(q.M) * q.srcs);
}

// The tile width of a problem and the estimated time of its schedule: rounds over the CTA
// pairs, each as long as a 128-deep stage's MMAs (0.6 us at 256 columns; narrower tiles run
// at 0.88 and 0.83 of the rate) or its operands' way into an SM: about 165 bytes a nanosecond
// (the large boxes of this kernel), half of that where rows do not start on 128-byte lines.
// At 256 a last round that fills at most half of the pairs runs as column halves, 0.53 of a
// whole one.
struct TilePlan {
  int bn = 256;
  int ctas = 0;
  double us = 1e30;
};

template <FfnOp kOp>
TilePlan tile_plan(const FfnProblem& q, int clusters) {
  bool lines = true;
  for (int i = 0; i < q.count_a; ++i) lines = lines && rows_aligned(q.A[i].ptr, q.A[i].ld, 2, 128);
  for (int i = 0; i < q.count_b; ++i) lines = lines && rows_aligned(q.B[i].ptr, q.B[i].ld, 2, 128);
  const double rate = lines ? 165e3 : 82e3;
  const double stages = static_cast<double>((q.K + kFfnKS - 1) / kFfnKS) * q.segs;
  const long long tiles_m = (q.M + BM - 1) / BM * q.srcs;
  constexpr int kWidths[] = {256, 192, 128};
  constexpr double kEff[] = {1.0, 0.88, 0.83};
  // 192 is built for linear_act alone: half of it is no whole number of epilogue boxes
  // (Gated) or of MN-major groups (the gradients, which would load a quarter more)
  auto built = [](int bn) { return bn != 192 || kOp == FfnOp::Linear; };
  const int width = tile_width_override();
  const bool forced = width == 256 || width == 128;
  TilePlan best;
  for (int i = 0; i < 3; ++i) {
    const int bn = kWidths[i], out_n = kOp == FfnOp::Gated ? bn / 2 : bn;
    if (!built(bn) || (forced && bn != width)) continue;
    const long long tiles = tiles_m * ((q.N + out_n - 1) / out_n);
    const long long full = tiles / clusters, rem = tiles % clusters;
    const bool halves = bn == 256 && rem > 0 && 2 * rem <= clusters;
    const double whole = std::max(0.6 * bn / 256 / kEff[i], (32768.0 + 128.0 * bn) / rate);
    const double half = std::max(0.32, 49152.0 / rate);
    const double busy = stages * (static_cast<double>(full) * whole +
                                  (rem == 0 ? 0.0 : (halves ? half : whole)));
    // streaming from DRAM takes CTAs: about 35 bytes a nanosecond each
    const double pairs = full > 0 ? clusters : static_cast<double>(halves ? 2 * rem : rem);
    const double dram = operand_bytes<kOp>(q) / std::min(kDramRate, 2.0 * pairs * 35e3);
    const double us = kUsFixed + 1.0 + std::max(busy, dram);
    if (us < best.us * 0.999) {
      best.bn = bn;
      best.ctas = 2 * static_cast<int>(full > 0 ? clusters : (halves ? 2 * rem : rem));
      best.us = us;
    }
  }
  return best;
}

// 256-row tiles: encodes the maps and launches.
template <FfnOp kOp>
int ffn_launch_tiles(const DeviceInfo& dev, const FfnProblem& q, int bn, cudaStream_t stream) {
  FfnParams p = {};
  p.M = static_cast<int>(q.M), p.N = static_cast<int>(q.N);
  p.kb_seg = static_cast<int>((q.K + kFfnKS - 1) / kFfnKS);
  p.segs = q.segs, p.srcs = q.srcs;
  p.late_wait = q.late_wait;
  p.bf16 = q.dtype == IGC_BF16;
  p.act = q.act;
  p.bias0 = q.bias[0], p.bias1 = q.bias[1], p.bias_f32 = q.bias_dtype == IGC_F32;
  p.R = q.R.ptr, p.ldr = q.R.ld, p.r_vec = rows_aligned(q.R.ptr, q.R.ld, 2, 16);
  FfnOperands ops = {};
  int rc = IGC_OK;
  for (int i = 0; i < q.count_a && rc == IGC_OK; ++i)
    rc = ffn_map_a(&ops.a[i], q, i, ffn_a_mn(kOp), ffn_a_mn(kOp) ? kFfnKS : BM_CTA);
  for (int i = 0; i < q.count_b && rc == IGC_OK; ++i)
    rc = ffn_map_b(&ops.b[i], q, i, ffn_b_mn(kOp), ffn_b_mn(kOp) ? kFfnKS : bn / 4);
  if (rc != IGC_OK) return rc;
  CUtensorMap out_maps[3] = {};
  for (int i = 0; i < 3; ++i) ffn_set_out(p, out_maps, i, q.out[i]);
  if constexpr (kOp == FfnOp::Linear)
    if (bn == 192) return ffn_launch_bn<kOp, 192>(dev, ops, out_maps, p, stream);
  return bn == 256 ? ffn_launch_bn<kOp, 256>(dev, ops, out_maps, p, stream)
                   : ffn_launch_bn<kOp, 128>(dev, ops, out_maps, p, stream);
}

// ---------------------------------------------------------------------------
// small outputs: 128-column blocks shared by clusters that split k
// ---------------------------------------------------------------------------
constexpr size_t kSmallSmemTwo = 110 * 1024;  // two CTAs on an SM
constexpr size_t kSmallSmemOne = 224 * 1024;

// Clusters of 1 .. kSkMaxSplit CTAs that run at once with one CTA on an SM (they stay
// within a GPC, whose SMs a larger cluster does not fill).
struct ClusterSlots {
  int clusters[kSkMaxSplit + 1];
};

// A GB300's 152 SMs, scaled to another number: what igc_plan_ffn works with.
inline ClusterSlots default_slots(int sms) {
  constexpr int k152[kSkMaxSplit + 1] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
  ClusterSlots s = {};
  for (int i = 1; i <= kSkMaxSplit; ++i) s.clusters[i] = std::max(1, k152[i] * sms / 152);
  return s;
}

struct SmallPlan {
  int m_blocks = 1, mt = 16, split = 1;
  double us = 1e30;
};

inline size_t small_stage_bytes(int mt) { return kSkWBytes + static_cast<size_t>(mt) * BK * 2; }
inline size_t small_part_bytes(int mt) { return static_cast<size_t>(mt) * kSkRows * 4; }
// Whether two CTAs with blocks of mt output rows fit on an SM with at least three stages each.
inline bool small_two_fit(int mt) {
  return small_part_bytes(mt) <= kSmallSmemTwo - 1024 &&
         3 * small_stage_bytes(mt) <= kSmallSmemTwo - 1024;
}

// What a CTA of the kernel takes: its 64-k blocks, ring stages, tensor-memory columns and
// dynamic shared memory.
struct SmallShape {
  int per_cta = 1, stages = 1;
  uint32_t tmem_cols = 32;
  size_t smem = 0;
};

inline SmallShape small_shape(int mt, int atoms, int split) {
  SmallShape s;
  while (s.tmem_cols < static_cast<uint32_t>(mt)) s.tmem_cols *= 2;
  s.per_cta = (atoms + split - 1) / split;
  const size_t stage = small_stage_bytes(mt);
  const size_t budget = (small_two_fit(mt) ? kSmallSmemTwo : kSmallSmemOne) - 1024;
  const size_t stages = std::min(std::min(budget / stage, static_cast<size_t>(kSkMaxStages)),
                                 static_cast<size_t>(s.per_cta));
  s.stages = static_cast<int>(stages);
  s.smem = std::max(1024 + std::max(stages * stage, small_part_bytes(mt)),
                    tmem_smem_floor(s.tmem_cols));
  return s;
}

// The number of output rows of a block and of CTAs that share one: the cheapest of the
// combinations.  Fewer rows and more CTAs mean more SMs at work on shorter parts, but W
// is read once per block of rows and each CTA's partial sums cross the cluster.
template <FfnOp kOp>
SmallPlan small_plan(const FfnProblem& q, int sms, const ClusterSlots& at_once) {
  constexpr int kOutT = kOp == FfnOp::Gated ? kSkRows / 2 : kSkRows;
  constexpr int kRowStep = ffn_a_mn(kOp) ? 64 : 16;
  const int atoms = static_cast<int>((q.K + BK - 1) / BK) * q.segs;
  const double unique = operand_bytes<kOp>(q);
  SmallPlan best;
  int last_mt = 0;
  for (int rows = kSkMaxMt; rows >= 32; rows -= 32) {
    const int64_t mb = (q.M + rows - 1) / rows;
    const int mt = static_cast<int>(((q.M + mb - 1) / mb + kRowStep - 1) / kRowStep * kRowStep);
    if (mt == last_mt || mt > kSkMaxMt || mb > 1 << 20) continue;
    last_mt = mt;
    const double blocks = static_cast<double>((q.N + kOutT - 1) / kOutT) *
                          static_cast<double>(mb) * q.srcs;
    for (int split = 1; split <= kSkMaxSplit && (split == 1 || atoms >= 2 * split); ++split) {
      if (split == 7) continue;  // (clusters of 7 waste a GPC's SMs as those of 8 do)
      const bool two = small_two_fit(mt);
      // (two to an SM, a cluster's CTAs find place more easily)
      const double alone = static_cast<double>(at_once.clusters[split] * split);
      const double slots = two ? 2.0 * sms * (split > 2 ? 0.9 : 1.0) : alone;
      const double ctas = blocks * split;
      const double waves = std::ceil(ctas / slots);
      const bool pairs = two && ctas > alone;  // two CTAs on some SMs
      const double rate = pairs ? kTwoCtaRate / 2 : (two ? kCtaRate : kDeepCtaRate);
      const double load =
          static_cast<double>((atoms + split - 1) / split) * BK * 2.0 * (kSkRows + mt) / rate;
      const double join =
          static_cast<double>(small_part_bytes(mt)) /
              (split > 1 ? (pairs ? kDsmemPerSm / 2 : kDsmemPerSm) : rate) +
          (split > 1 ? 0.3 : 0.0);
      const double streams = ctas / waves;
      const double dram = unique / (kDramMost * streams / (streams + 70.0));
      const double busy = std::max(waves * load, dram);
      const double us = kUsFixed + busy + waves * join + (waves - 1.0) * kUsWave;
      if (us < best.us) {
        best.m_blocks = static_cast<int>(mb);
        best.mt = mt;
        best.split = split;
        best.us = us;
      }
    }
  }
  return best;
}

// Sets the kernel's shared-memory attribute and asks how many of its clusters run at once
// (cached per device).
template <FfnOp kOp>
int small_setup(const DeviceInfo& dev, const ClusterSlots** slots) {
  static std::once_flag once[64];
  static int rcs[64];
  static ClusterSlots table[64];
  const int d = dev.device;
  std::call_once(once[d], [&] {
    auto kern = igc_ffn_small_kernel<kOp>;
    rcs[d] = IGC_ERR_CUDA;
    if (dev.smem_optin < kSmallSmemOne + 1024) {
      rcs[d] = IGC_ERR_UNSUPPORTED;
      return;
    }
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmallSmemOne)) != cudaSuccess)
      return;
    table[d] = default_slots(dev.sm_count);
    for (int s = 2; s <= kSkMaxSplit; ++s) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(s * dev.sm_count), 1, 1);
      cfg.blockDim = dim3(kSkThreads, 1, 1);
      cfg.dynamicSmemBytes = kSmallSmemOne;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = static_cast<unsigned>(s);
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0)
        table[d].clusters[s] = n;
      else
        (void)cudaGetLastError();
    }
    rcs[d] = IGC_OK;
  });
  *slots = &table[d];
  return rcs[d];
}

template <FfnOp kOp>
int ffn_launch_small(const DeviceInfo& dev, const FfnProblem& q, const ProductPlan& plan,
                     cudaStream_t stream) {
  auto kern = igc_ffn_small_kernel<kOp>;
  constexpr int kOutT = kOp == FfnOp::Gated ? kSkRows / 2 : kSkRows;
  SmallParams p = {};
  p.M = static_cast<int>(q.M), p.N = static_cast<int>(q.N);
  p.m_blocks = plan.m_blocks;
  p.mt = plan.mt;
  p.atoms_seg = static_cast<int>((q.K + BK - 1) / BK);
  p.atoms = p.atoms_seg * q.segs;
  const long long blocks = (q.N + kOutT - 1) / kOutT * p.m_blocks * q.srcs;
  p.split = plan.split;
  if (blocks * p.split > 0x7fffffffLL) return IGC_ERR_UNSUPPORTED;
  const SmallShape shape = small_shape(p.mt, p.atoms, p.split);
  p.per_cta = shape.per_cta, p.stages = shape.stages, p.tmem_cols = shape.tmem_cols;
  p.late_wait = q.late_wait;
  // Weights past half of the L2 are gone before they are read again: marked to be evicted
  // first, they leave the lines that the next kernel prefetches alone (134 MB, one token:
  // 22.7 -> 21.1 us; smaller weights, which may still be there next time, are not marked).
  p.once = p.m_blocks == 1 &&
           2.0 * static_cast<double>(q.N) * static_cast<double>(q.K) * q.count_b >= 64e6;
  p.bf16 = q.dtype == IGC_BF16;
  p.act = q.act;
  p.bias0 = q.bias[0], p.bias1 = q.bias[1], p.bias_f32 = q.bias_dtype == IGC_F32;
  p.R = q.R.ptr, p.ldr = q.R.ld, p.r_vec = rows_aligned(q.R.ptr, q.R.ld, 2, 8);
  p.wait_limit_ns = wait_limit_ns();
  p.status = status_word();
  for (int i = 0; i < 3; ++i) {
    const size_t es = elem_size(q.out[i].dtype);
    p.out[i] = const_cast<void*>(q.out[i].ptr);
    p.ld[i] = q.out[i].ld;
    p.f32[i] = q.out[i].dtype == IGC_F32;
    p.vec[i] = rows_aligned(q.out[i].ptr, q.out[i].ld, es, 4 * es);
  }
  // the kernel's A operand is the problem's B (the output's columns) and the other way round
  CUtensorMap ma[2] = {}, mb[2] = {};
  int rc = IGC_OK;
  for (int i = 0; i < q.count_b && rc == IGC_OK; ++i)
    rc = ffn_map_b(&ma[i], q, i, ffn_b_mn(kOp), ffn_b_mn(kOp) ? BK : kOutT);
  for (int i = 0; i < q.count_a && rc == IGC_OK; ++i)
    rc = ffn_map_a(&mb[i], q, i, ffn_a_mn(kOp), ffn_a_mn(kOp) ? BK : p.mt);
  if (rc != IGC_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks * p.split), 1, 1);
  cfg.blockDim = dim3(kSkThreads, 1, 1);
  cfg.dynamicSmemBytes = shape.smem;
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
  if (cudaLaunchKernelEx(&cfg, kern, ma[0], ma[1], mb[0], mb[1], p) != cudaSuccess) {
    (void)cudaGetLastError();
    return IGC_ERR_CUDA;
  }
  return IGC_OK;
}

// Which of the two kernels runs a problem: the one with the shorter estimate, unless the
// calling thread forced a tile width (igc_set_tile_width).
inline ProductPlan join_plans(const SmallPlan& small, const TilePlan& tiles) {
  ProductPlan p;
  p.small = small.us < tiles.us && tile_width_override() == 0;
  p.mt = small.mt, p.m_blocks = small.m_blocks, p.split = small.split;
  p.bn = tiles.bn, p.tile_ctas = tiles.ctas;
  p.small_us = small.us, p.tiles_us = tiles.us;
  return p;
}

template <FfnOp kOp>
int ffn_plan(const DeviceInfo& dev, const FfnProblem& q, ProductPlan* plan) {
  int clusters = 0;
  int rc = ffn_kernel_setup<kOp, 256>(dev, &clusters);
  if (rc != IGC_OK) return rc;
  const ClusterSlots* slots = nullptr;
  rc = small_setup<kOp>(dev, &slots);
  if (rc != IGC_OK) return rc;
  *plan = join_plans(small_plan<kOp>(q, dev.sm_count, *slots), tile_plan<kOp>(q, clusters));
  return IGC_OK;
}

template <FfnOp kOp>
int ffn_launch(const DeviceInfo& dev, const FfnProblem& q, const ProductPlan& plan,
               cudaStream_t stream) {
  return plan.small ? ffn_launch_small<kOp>(dev, q, plan, stream)
                    : ffn_launch_tiles<kOp>(dev, q, plan.bn, stream);
}

// The plan of a product on a GPU of `sms` SMs.
template <FfnOp kOp>
ProductPlan ffn_plan_host(const FfnProblem& q, int sms) {
  return join_plans(small_plan<kOp>(q, sms, default_slots(sms)), tile_plan<kOp>(q, sms / 2));
}

// It in igc_plan_ffn's form (see igc_ffn.h).
inline void ffn_plan_out(const FfnProblem& q, const ProductPlan& p, int32_t* out) {
  out[0] = p.small;
  out[1] = p.small ? p.mt : BM;
  out[2] = p.small ? p.m_blocks : static_cast<int32_t>((q.M + BM - 1) / BM);
  out[3] = p.small ? kSkRows : p.bn;
  out[4] = p.small ? p.split : 1;
  out[5] = static_cast<int32_t>(std::min(p.small_us * 1000, 2e9));
  out[6] = static_cast<int32_t>(std::min(p.tiles_us * 1000, 2e9));
}

// Tensor-memory columns and dynamic shared memory of a CTA of that product's kernel.
template <FfnOp kOp>
void ffn_resources_host(const FfnProblem& q, const ProductPlan& p, int32_t* out) {
  if (p.small) {
    const int atoms = static_cast<int>((q.K + BK - 1) / BK) * q.segs;
    const SmallShape s = small_shape(p.mt, atoms, p.split);
    out[0] = static_cast<int32_t>(s.tmem_cols), out[1] = static_cast<int32_t>(s.smem);
  } else if (p.bn == 256) {
    out[0] = FfnCfg<kOp, 256>::kTmemCols, out[1] = FfnCfg<kOp, 256>::kSmemBytes;
  } else if (p.bn == 128) {
    out[0] = FfnCfg<kOp, 128>::kTmemCols, out[1] = FfnCfg<kOp, 128>::kSmemBytes;
  } else if constexpr (kOp == FfnOp::Linear) {
    out[0] = FfnCfg<kOp, 192>::kTmemCols, out[1] = FfnCfg<kOp, 192>::kSmemBytes;
  }
}

}  // namespace igc
