// The feed-forward products where 256-row tiles would leave most of the GPU idle: few
// rows of X (decode) and small matrices.  tcgen05 with the operands' places swapped:
//
//   out[m, n] = sum_k B[m, k] A[n, k]
//
// 128 output columns (rows of W in the forward pass) are the A operand of the MMA
// (M = 128), up to 256 output rows, padded to a multiple of 16, its B operand (N).  With
// few rows the weights are the work: each of them is used once, and the kernel is a
// stream of W at memory speed: TMA copies 64-deep stages of a CTA's part of W through a
// ring; X is small and comes from L2.  For the gated pair, 64 rows of Wg and the same 64
// rows of Wu make up the 128.  The gradients' operands are contiguous along the output
// (MN-major atoms: 64 outputs of every k, see ffn_tc.cuh).
//
// There are too few such blocks to fill the GPU, so a cluster of S CTAs shares one: CTA r
// takes the r-th part of k, writes its fp32 partial sums to its own shared memory, and
// after a cluster barrier every CTA adds up a share of the outputs over the S partial sums
// (distributed shared memory, in the order of r: no atomics, no workspace, the same
// result every time) and applies the epilogue.
//
// What bounds it: DRAM for few rows (one token through 4096 x 16384 bf16 weights, 134 MB:
// 21.2 us back to back, 6.3 TB/s; gated 48 x 16384 x 4096, 268 MB: 43.7 us), the SMs' intake
// from L2 from some 64 rows on, where X weighs as much as W (128 x 8192 x 8192: 27.8 us),
// and latency for small outputs (333 x 1000 x 2056: 10 us).
#pragma once

#include "ffn_act.cuh"
#include "ffn_tc.cuh"

namespace igc {

constexpr int kSkThreads = 256;
constexpr int kSkRows = 128;                             // output columns of a block (MMA's M)
constexpr uint32_t kSkWBytes = kSkRows * BK * 2;         // 16 KB per stage
constexpr uint32_t kSkGroup = 64 * BK * 2;               // an MN-major atom: 64 outputs x 64 k
constexpr int kSkMaxMt = 256;                            // output rows of a block (MMA's N)
constexpr int kSkMaxStages = 12;
constexpr int kSkMaxSplit = 8;                           // portable cluster size

struct SmallParams {
  int M, N;        // rows and columns of one output matrix
  int mt;          // output rows of a block: a multiple of 16 (of 64 for GradW)
  int m_blocks;    // blocks of rows of one output matrix (GradW: of each of the two)
  int atoms_seg;   // 64-k blocks of one contraction segment
  int atoms;       // of all segments
  int per_cta;     // of which each CTA takes this many
  int split;       // CTAs of a cluster
  int stages;
  int once;        // the A operand is read once and does not fit L2: evict it first
  uint32_t tmem_cols;
  int bf16, act;
  int late_wait;   // see ffn_dependency_wait
  const void* bias0;
  const void* bias1;
  int bias_f32;
  const void* R;
  long long ldr;
  int r_vec;       // rows of R / out[i] take 8-byte (16-bit) or 16-byte (fp32) accesses
  void* out[3];    // as FfnParams::out
  long long ld[3];
  int f32[3], vec[3];
  unsigned long long wait_limit_ns;
  unsigned long long* status;
};

enum : uint32_t { kSiteSkEmpty = 16, kSiteSkFull = 17, kSiteSkDone = 18 };

// Stores 4 consecutive results of row m from column n.
__device__ __forceinline__ void sk_store4(const SmallParams& p, int slot, int m, int n,
                                          const float (&v)[4]) {
  const bool whole = p.vec[slot] && n + 4 <= p.N;
  const long long at = static_cast<long long>(m) * p.ld[slot] + n;
  if (p.f32[slot]) {
    float* o = static_cast<float*>(p.out[slot]) + at;
    if (whole) {
      *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      for (int i = 0; i < 4; ++i)
        if (n + i < p.N) o[i] = v[i];
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(p.out[slot]) + at;
    if (whole) {
      *reinterpret_cast<uint2*>(o) =
          make_uint2(pack16(v[0], v[1], p.bf16), pack16(v[2], v[3], p.bf16));
    } else {
      for (int i = 0; i < 4; ++i)
        if (n + i < p.N) store16(o, i, v[i], p.bf16);
    }
  }
}

__device__ __forceinline__ void sk_add_bias4(const SmallParams& p, const void* bias, int n,
                                             float (&v)[4]) {
  if (bias == nullptr) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < p.N) v[i] += load_vec(bias, n + i, p.bias_f32, p.bf16);
}

// One stage's copies: 64 k of the block's 128 output columns and mt output rows.
template <FfnOp kOp>
__device__ __forceinline__ void sk_load_stage(const SmallParams& p, const CUtensorMap* tmA0,
                                              const CUtensorMap* tmA1, const CUtensorMap* tmB,
                                              uint8_t* dst, uint64_t* bar, int k, int n_blk,
                                              int m_blk, uint64_t policy) {
  uint8_t* b_dst = dst + kSkWBytes;
  if constexpr (ffn_b_mn(kOp)) {  // A is contiguous along the output columns
    tma_load_2d(dst, tmA0, bar, n_blk, k);
    tma_load_2d(dst + kSkGroup, tmA0, bar, n_blk + 64, k);
  } else if constexpr (kOp == FfnOp::Gated) {
    if (p.once) {
      tma_load_2d_hint(dst, tmA0, bar, k, n_blk, policy);
      tma_load_2d_hint(dst + kSkWBytes / 2, tmA1, bar, k, n_blk, policy);
    } else {
      tma_load_2d(dst, tmA0, bar, k, n_blk);
      tma_load_2d(dst + kSkWBytes / 2, tmA1, bar, k, n_blk);
    }
  } else if (p.once) {
    tma_load_2d_hint(dst, tmA0, bar, k, n_blk, policy);
  } else {
    tma_load_2d(dst, tmA0, bar, k, n_blk);
  }
  if constexpr (ffn_a_mn(kOp)) {  // B is contiguous along the output rows
    for (int g = 0; g < p.mt / 64; ++g)
      tma_load_2d(b_dst + g * kSkGroup, tmB, bar, m_blk + 64 * g, k);
  } else {
    tma_load_2d(b_dst, tmB, bar, k, m_blk);
  }
}

template <FfnOp kOp, int kSplit, int kSteps>
__device__ __forceinline__ void sk_outputs(const SmallParams& p, const float* part, int rank,
                                           int rows, int m_blk, int n_blk, int src) {
  constexpr int kOutT = kOp == FfnOp::Gated ? kSkRows / 2 : kSkRows;
  constexpr int kParts = kOp == FfnOp::Gated ? 2 : 1;  // G and U
  uint32_t peer[kSplit];
#pragma unroll
  for (int r = 0; r < kSplit; ++r)
    peer[r] = mapa_shared(smem_u32(part), static_cast<uint32_t>(r < p.split ? r : 0));
  const int steps = rows * (kOutT / 4);
  const int stride = p.split * kSkThreads;
  for (int first = rank * kSkThreads + static_cast<int>(threadIdx.x); first < steps;
       first += kSteps * stride) {
    float v[kSteps][kParts][4];
    uint2 res[kSteps];
    const bool whole_r = kOp == FfnOp::Linear && p.R != nullptr && p.r_vec;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const int it = first + j * stride;
      if (it >= steps) continue;
      const int row = it / (kOutT / 4), w = it % (kOutT / 4) * 4;
      if (whole_r && n_blk + w + 4 <= p.N)
        res[j] = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.R) +
                                                 static_cast<long long>(m_blk + row) * p.ldr +
                                                 n_blk + w);
#pragma unroll
      for (int h = 0; h < kParts; ++h) {
        const uint32_t off = static_cast<uint32_t>(row * kSkRows + w + h * kOutT) * 4u;
        float4 q[kSplit];
#pragma unroll
        for (int r = 0; r < kSplit; ++r)
          if (r < p.split) q[r] = ld_shared_cluster_f32x4(peer[r] + off);
        v[j][h][0] = q[0].x, v[j][h][1] = q[0].y, v[j][h][2] = q[0].z, v[j][h][3] = q[0].w;
#pragma unroll
        for (int r = 1; r < kSplit; ++r)
          if (r < p.split)
            v[j][h][0] += q[r].x, v[j][h][1] += q[r].y, v[j][h][2] += q[r].z,
                v[j][h][3] += q[r].w;
      }
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const int it = first + j * stride;
      if (it >= steps) continue;
      const int row = it / (kOutT / 4), w = it % (kOutT / 4) * 4;
      const int m = m_blk + row, n = n_blk + w;
      if (n >= p.N) continue;
      float(&y)[4] = v[j][0];
      if constexpr (kOp == FfnOp::Gated) {
        float(&u)[4] = v[j][kParts - 1];
        sk_add_bias4(p, p.bias0, n, y);
        sk_add_bias4(p, p.bias1, n, u);
        if (p.out[1] != nullptr) {
          sk_store4(p, 1, m, n, y);
          sk_store4(p, 2, m, n, u);
        }
        with_act(p.act, [&](auto a) {
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = act_f32<decltype(a)::value>(y[i]) * u[i];
        });
      } else if constexpr (kOp == FfnOp::Linear) {
        sk_add_bias4(p, p.bias0, n, y);
        if (p.out[1] != nullptr) sk_store4(p, 1, m, n, y);
        with_act(p.act, [&](auto a) {
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = act_f32<decltype(a)::value>(y[i]);
        });
        if (whole_r && n + 4 <= p.N) {
          const float2 lo = unpack16(res[j].x, p.bf16), hi = unpack16(res[j].y, p.bf16);
          y[0] += lo.x, y[1] += lo.y, y[2] += hi.x, y[3] += hi.y;
        } else if (p.R != nullptr) {
          const uint16_t* r =
              static_cast<const uint16_t*>(p.R) + static_cast<long long>(m) * p.ldr + n;
          for (int i = 0; i < 4; ++i)
            if (n + i < p.N) y[i] += load16(r, i, p.bf16);
        }
      }
      sk_store4(p, kOp == FfnOp::GradW ? src : 0, m, n, y);
    }
  }
}

// kOp's operands as in ffn_tc.cuh, with the places swapped: tmA* hold the matrix whose
// index is the output column (W; X for GradW), tmB* the other (X; D for the gradients).
template <FfnOp kOp>
__global__ void __launch_bounds__(kSkThreads)
    igc_ffn_small_kernel(const __grid_constant__ CUtensorMap tmA0,
                         const __grid_constant__ CUtensorMap tmA1,
                         const __grid_constant__ CUtensorMap tmB0,
                         const __grid_constant__ CUtensorMap tmB1, const SmallParams p) {
  constexpr bool kGated = kOp == FfnOp::Gated;
  constexpr int kOutT = kGated ? kSkRows / 2 : kSkRows;  // output columns of a block
  constexpr bool kAMn = ffn_b_mn(kOp), kBMn = ffn_a_mn(kOp);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t stage_bytes = kSkWBytes + static_cast<uint32_t>(p.mt) * (BK * 2);
  float* part = reinterpret_cast<float*>(smem);  // over the ring, once it is drained
  __shared__ uint64_t full[kSkMaxStages], empty[kSkMaxStages], done;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 32, 0);
  const int lane = static_cast<int>(lane_id());
  const int rank = static_cast<int>(cluster_ctarank());
  // row blocks of one column block are neighbours: they share its weights in L2
  const int blk = static_cast<int>(blockIdx.x) / p.split;
  const int m_all = p.m_blocks * (kOp == FfnOp::GradW && p.out[1] != nullptr ? 2 : 1);
  const int mb = blk % m_all;
  const int src = kOp == FfnOp::GradW ? mb / p.m_blocks : 0;
  const int m_blk = (mb - src * p.m_blocks) * p.mt;
  const int rows = min(p.mt, p.M - m_blk);
  const int n_blk = (blk / m_all) * kOutT;
  const int a0 = rank * p.per_cta;
  const int n_atoms = max(0, min(p.per_cta, p.atoms - a0));
  const uint64_t lim = p.wait_limit_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA0);
    tma_prefetch_desc(&tmB0);
    if (kGated) tma_prefetch_desc(&tmA1);
  }
  if (warp == 1) {
    tmem_alloc_1cta(&tmem_slot, p.tmem_cols);
    tmem_relinquish_1cta();
  }
  // While the previous kernel in the stream finishes: the first stages of the weights
  // into L2 (a hint that makes nothing visible, so it may come before the wait below).
  // Measured on one token through 4096 x 16384 bf16 weights: 23.1 us without it, 21.1 with
  // one ring's depth, 21.9 and 25.7 with 16 and 32 stages (the bursts delay the kernel
  // that is still running).
  if constexpr (kOp == FfnOp::Linear || kOp == FfnOp::Gated) {
    if (warp == 2 && lane == 0) {
      for (int i = 0; i < n_atoms && i < p.stages; ++i) {
        tma_prefetch_2d(&tmA0, (a0 + i) * BK, n_blk);
        if (kGated) tma_prefetch_2d(&tmA1, (a0 + i) * BK, n_blk);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  ffn_dependency_wait(p.late_wait);
  const uint32_t tmem = tmem_slot;

  if (warp == 0 && lane == 0) {
    const uint64_t policy = policy_evict_first();
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;
    for (; issued < n_atoms; ++issued) {
      if (!mbar_wait(&empty[stage], phase ^ 1u, lim, &abort_flag, p.status, kSiteSkEmpty)) break;
      const int seg = kOp == FfnOp::GradX ? (a0 + issued) / p.atoms_seg : 0;
      const CUtensorMap* mapA = seg ? &tmA1 : &tmA0;
      const CUtensorMap* mapB = (kOp == FfnOp::GradX ? seg : src) ? &tmB1 : &tmB0;
      mbar_arrive_expect_tx(&full[stage], stage_bytes);
      sk_load_stage<kOp>(p, mapA, &tmA1, mapB, smem + static_cast<uint32_t>(stage) * stage_bytes,
                         &full[stage], (a0 + issued - seg * p.atoms_seg) * BK, n_blk, m_blk,
                         policy);
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    // after an abort, the copies in flight get time to land before the CTA may exit
    if (*static_cast<volatile int*>(&abort_flag))
      drain_fills(full, p.stages, stage, phase, issued, lim);
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = make_idesc_kind_f16(kSkRows, p.mt, p.bf16 ? 1u : 0u) |
                           (kAMn ? 1u << 15 : 0u) | (kBMn ? 1u << 16 : 0u);
    // 16 k: two 8-k groups of an MN-major atom, 32 bytes of a K-major row
    constexpr uint32_t kStepA = kAMn ? 2048u : 32u, kStepB = kBMn ? 2048u : 32u;
    int stage = 0;
    uint32_t phase = 0;
    for (int i = 0; i < n_atoms; ++i) {
      if (!mbar_wait(&full[stage], phase, lim, &abort_flag, p.status, kSiteSkFull)) break;
      tc_fence_after();
      const uint32_t w = smem_u32(smem) + static_cast<uint32_t>(stage) * stage_bytes;
      const uint64_t ad = kAMn ? make_sw128_mnmajor_desc(w, kSkGroup) : make_sw128_kmajor_desc(w);
      const uint64_t bd = kBMn ? make_sw128_mnmajor_desc(w + kSkWBytes, kSkGroup)
                               : make_sw128_kmajor_desc(w + kSkWBytes);
#pragma unroll
      for (int k = 0; k < BK / 16; ++k)
        umma_f16_ss_1cta(tmem, ad + ((k * kStepA) >> 4), bd + ((k * kStepB) >> 4), idesc,
                         (i > 0 || k > 0) ? 1u : 0u);
      umma_commit_1cta(&empty[stage]);
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    umma_commit_1cta(&done);
  }
  __syncwarp();

  // Partial sums to shared memory: part[m][w] for output row m and column w of the block.
  // The MMAs are done (so every copy has landed and been read): the ring is free.
  const bool ok = __all_sync(0xffffffffu, mbar_wait(&done, 0, lim, &abort_flag, p.status,
                                                    kSiteSkDone));
  tc_fence_after();
  if (ok) {
    const int quad = warp & 3;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    for (int c = (warp >> 2) * 16; c < rows; c += 32) {
      uint32_t r[16];
      if (n_atoms > 0) {
        tmem_ld_32x32b_x16(taddr + static_cast<uint32_t>(c), r);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = 0u;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (c + i < rows)
          part[(c + i) * kSkRows + quad * 32 + lane] = __uint_as_float(r[i]);
    }
  }
  // The columns go back before anything is waited for in another CTA: no CTA of this kernel
  // holds columns while it needs one that may itself still be waiting for some.
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_1cta(tmem, p.tmem_cols);
  }
  if (p.split > 1) cluster_sync();

  // Outputs: 4 columns per step, the steps dealt over the cluster's threads.  A thread
  // takes several steps at a time (more of them where few partial sums are added), so that
  // their shared-memory and residual loads overlap.
  if (ok) {
    if (p.split > 2)
      sk_outputs<kOp, kSkMaxSplit, 2>(p, part, rank, rows, m_blk, n_blk, src);
    else
      sk_outputs<kOp, 2, 4>(p, part, rank, rows, m_blk, n_blk, src);
  }
  // no CTA may exit while another one still reads its partial sums
  if (p.split > 1) cluster_sync();
  ffn_dependency_end(p.late_wait);
}

}  // namespace igc
