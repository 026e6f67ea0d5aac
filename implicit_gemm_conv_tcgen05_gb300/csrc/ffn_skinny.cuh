// The feed-forward products for few rows of X (decode): Y^T = W X^T on tcgen05.
//
// With few rows the weights are the work: N K elements that are used once each, so
// the kernel is a stream of W at memory speed.  The operands therefore swap places:
// 128 rows of W are the A operand of the MMA (M = 128) and the rows of X, padded to a
// multiple of 16, are its B operand (N = 16 .. 128); a CTA accumulates 128 weight rows
// x all X rows in tensor memory while TMA streams its part of W through a ring of
// 64-deep stages.  X is small and comes from L2.  For the gated pair, 64 rows of Wg
// and the same 64 rows of Wu make up the 128.
//
// A layer has too few 128-row blocks to fill the GPU, so a cluster of S CTAs shares a
// block: CTA r takes the r-th part of k, writes its fp32 partial sums to its own
// shared memory, and after a cluster barrier every CTA adds up a share of the outputs
// over the S partial sums (distributed shared memory, in the order of r: no atomics,
// no workspace, the same result every time) and applies the epilogue.
#pragma once

#include "ffn_act.cuh"
#include "gemm_tc.cuh"

namespace igc {

constexpr int kSkThreads = 256;
constexpr int kSkRows = 128;                             // weight rows of a block
constexpr uint32_t kSkWBytes = kSkRows * BK * 2;         // 16 KB per stage
constexpr int kSkMaxStages = 12;
constexpr int kSkMaxSplit = 8;                           // portable cluster size

struct SkinnyParams {
  int M, N;        // rows of X (at most mt), output columns
  int mt;          // rows of X padded to a multiple of 16: the MMA's N
  int atoms;       // 64-k blocks
  int per_cta;     // of which each CTA takes this many
  int split;       // CTAs of a cluster
  int stages;
  uint32_t tmem_cols;
  int bf16, act;
  const void* bias0;
  const void* bias1;
  int bias_f32;
  const void* R;
  long long ldr;
  int r_vec;       // rows of R / out[i] take 8-byte (16-bit) or 16-byte (fp32) accesses
  void* out[3];    // Linear: Y, Z; Gated: H, G, U
  long long ld[3];
  int f32[3], vec[3];
  unsigned long long wait_limit_ns;
  unsigned long long* status;
};

enum : uint32_t { kSiteSkEmpty = 16, kSiteSkFull = 17, kSiteSkDone = 18 };

// Stores 4 consecutive results of row m from column n.
__device__ __forceinline__ void sk_store4(const SkinnyParams& p, int slot, int m, int n,
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

__device__ __forceinline__ void sk_add_bias4(const SkinnyParams& p, const void* bias, int n,
                                             float (&v)[4]) {
  if (bias == nullptr) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < p.N) v[i] += load_vec(bias, n + i, p.bias_f32, p.bf16);
}

template <bool kGated>
__global__ void __launch_bounds__(kSkThreads)
    igc_ffn_skinny_kernel(const __grid_constant__ CUtensorMap tmX,
                          const __grid_constant__ CUtensorMap tmW0,
                          const __grid_constant__ CUtensorMap tmW1, const SkinnyParams p) {
  constexpr int kOutT = kGated ? kSkRows / 2 : kSkRows;  // output columns of a block

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
  const int n_blk = (static_cast<int>(blockIdx.x) / p.split) * kOutT;
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
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW0);
    if (kGated) tma_prefetch_desc(&tmW1);
  }
  if (warp == 1) {
    tmem_alloc_1cta(&tmem_slot, p.tmem_cols);
    tmem_relinquish_1cta();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();
  grid_dependents_launch();
  const uint32_t tmem = tmem_slot;

  if (warp == 0 && lane == 0) {
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;
    for (; issued < n_atoms; ++issued) {
      if (!mbar_wait(&empty[stage], phase ^ 1u, lim, &abort_flag, p.status, kSiteSkEmpty)) break;
      uint8_t* dst = smem + static_cast<uint32_t>(stage) * stage_bytes;
      const int k = (a0 + issued) * BK;
      mbar_arrive_expect_tx(&full[stage], stage_bytes);
      if (kGated) {
        tma_load_2d(dst, &tmW0, &full[stage], k, n_blk);
        tma_load_2d(dst + kSkWBytes / 2, &tmW1, &full[stage], k, n_blk);
      } else {
        tma_load_2d(dst, &tmW0, &full[stage], k, n_blk);
      }
      tma_load_2d(dst + kSkWBytes, &tmX, &full[stage], k, 0);
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    // after an abort, the copies in flight get time to land before the CTA may exit
    if (*static_cast<volatile int*>(&abort_flag))
      drain_fills(full, p.stages, stage, phase, issued, lim);
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = make_idesc_kind_f16(kSkRows, p.mt, p.bf16 ? 1u : 0u);
    int stage = 0;
    uint32_t phase = 0;
    for (int i = 0; i < n_atoms; ++i) {
      if (!mbar_wait(&full[stage], phase, lim, &abort_flag, p.status, kSiteSkFull)) break;
      tc_fence_after();
      const uint32_t w = smem_u32(smem) + static_cast<uint32_t>(stage) * stage_bytes;
      const uint64_t wd = make_sw128_kmajor_desc(w);
      const uint64_t xd = make_sw128_kmajor_desc(w + kSkWBytes);
#pragma unroll
      for (int k = 0; k < BK / 16; ++k)
        umma_f16_ss_1cta(tmem, wd + ((k * 32) >> 4), xd + ((k * 32) >> 4), idesc,
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

  // Partial sums to shared memory: part[m][w] for row m of X and weight row w of the
  // block.  The MMAs are done (so every copy has landed and been read): the ring is free.
  const bool ok = __all_sync(0xffffffffu, mbar_wait(&done, 0, lim, &abort_flag, p.status,
                                                    kSiteSkDone));
  tc_fence_after();
  if (ok) {
    const int quad = warp & 3;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    for (int c = (warp >> 2) * 16; c < p.M; c += 32) {
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
        if (c + i < p.M)
          part[(c + i) * kSkRows + quad * 32 + lane] = __uint_as_float(r[i]);
    }
  }
  tc_fence_before();
  if (p.split > 1)
    cluster_sync();
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_1cta(tmem, p.tmem_cols);
  }

  // Outputs: 4 columns per step, the steps dealt over the cluster's threads.
  if (ok) {
    uint32_t src[kSkMaxSplit];
#pragma unroll
    for (int r = 0; r < kSkMaxSplit; ++r)
      src[r] = r < p.split ? mapa_shared(smem_u32(part), static_cast<uint32_t>(r)) : 0u;
    auto sum4 = [&](int m, int w, float(&v)[4]) {
      const uint32_t off = static_cast<uint32_t>(m * kSkRows + w) * 4u;
      float4 q[kSkMaxSplit];
#pragma unroll
      for (int r = 0; r < kSkMaxSplit; ++r)
        if (r < p.split) q[r] = ld_shared_cluster_f32x4(src[r] + off);
      v[0] = q[0].x, v[1] = q[0].y, v[2] = q[0].z, v[3] = q[0].w;
#pragma unroll
      for (int r = 1; r < kSkMaxSplit; ++r)
        if (r < p.split) v[0] += q[r].x, v[1] += q[r].y, v[2] += q[r].z, v[3] += q[r].w;
    };
    const int steps = p.M * (kOutT / 4);
    for (int it = rank * kSkThreads + static_cast<int>(threadIdx.x); it < steps;
         it += p.split * kSkThreads) {
      const int m = it / (kOutT / 4);
      const int w = (it - m * (kOutT / 4)) * 4;
      const int n = n_blk + w;
      if (n >= p.N) continue;
      float v[4];
      sum4(m, w, v);
      sk_add_bias4(p, p.bias0, n, v);
      if constexpr (kGated) {
        float u[4];
        sum4(m, w + kOutT, u);
        sk_add_bias4(p, p.bias1, n, u);
        if (p.out[1] != nullptr) {
          sk_store4(p, 1, m, n, v);
          sk_store4(p, 2, m, n, u);
        }
        with_act(p.act, [&](auto a) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = act_f32<decltype(a)::value>(v[i]) * u[i];
        });
      } else {
        if (p.out[1] != nullptr) sk_store4(p, 1, m, n, v);
        with_act(p.act, [&](auto a) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = act_f32<decltype(a)::value>(v[i]);
        });
        if (p.R != nullptr) {
          const uint16_t* row =
              static_cast<const uint16_t*>(p.R) + static_cast<long long>(m) * p.ldr + n;
          if (p.r_vec && n + 4 <= p.N) {
            const uint2 q = *reinterpret_cast<const uint2*>(row);
            const float2 lo = unpack16(q.x, p.bf16), hi = unpack16(q.y, p.bf16);
            v[0] += lo.x, v[1] += lo.y, v[2] += hi.x, v[3] += hi.y;
          } else {
            for (int i = 0; i < 4; ++i)
              if (n + i < p.N) v[i] += load16(row, i, p.bf16);
          }
        }
      }
      sk_store4(p, 0, m, n, v);
    }
  }
  // no CTA may exit while another one still reads its partial sums
  if (p.split > 1) cluster_sync();
}

}  // namespace igc
