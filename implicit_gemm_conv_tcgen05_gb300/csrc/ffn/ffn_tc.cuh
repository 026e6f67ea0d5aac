// Persistent tcgen05 GEMM of the feed-forward operators (sm_103a, 2-CTA tiles).
//
//   Linear : Z = X W^T + bias, Y = act(Z) + R       operands contiguous along k
//   Gated  : H = act(X Wg^T + bg) * (X Wu^T + bu)   operands contiguous along k
//   GradX  : dX = sum_s D_s W_s                     W_s contiguous along the output column
//   GradW  : dW_s = D_s^T X                         both contiguous along the output
//
// where D_s is the gradient of the pre-activation(s): s runs over one matrix for
// linear_act and over two (dG, dU) for gated_ffn, whose two products of dX are one
// contraction of twice the length and whose two weight gradients are one launch.
//
// A cluster of two CTAs computes one 256 x BN accumulator tile with
// tcgen05.mma.cta_group::2: CTA r holds rows [128 r, 128 r + 128) of the A tile and
// rows [BN/2 r, BN/2 (r+1)) of the B tile, and gets its 128 x BN accumulator in its
// own tensor memory.  For Gated, CTA 0's half of the B tile comes from Wg and CTA
// 1's from Wu, over the same BN/2 output columns: each CTA's accumulator then holds
// G in its first BN/2 columns and U in the others, and the thread that owns an
// output row reads both.
//
// Operands are staged by TMA in 128-byte swizzle atoms.  Contiguous along k
// ("K-major"): an atom is 64 k of every row, rows of 128 bytes.  Contiguous along
// the output dimension ("MN-major"): an atom is 64 outputs of every k, k rows of
// 128 bytes, so that no operand is ever transposed in memory; the matrix descriptor
// and the instruction descriptor say which of the two it is.
//
// What bounds it: the tensor cores.  At 256 columns a stage's MMAs take as long as its
// operands' 64 KB need into an SM (64 bytes a clock), so no narrower tile keeps the rate
// and every box that the epilogue moves through shared memory costs the main loop a little.
// Measured (bf16, bursts): 8192^3 without an epilogue 565 us, 1945 TFLOP/s (the vendor
// library 558); tanh-GELU + 4, residual + 13, Z kept + 17.  Gated 8192 x 16384 x 4096 with G
// and U kept 1132 us, 1943 TFLOP/s (the vendor's product alone 1090); its dX and dW 1120 us each.
// Under the power limit of a long run: 687 to 706, 1279 to 1318 and 2795 to 2887 us (the whole
// backward pass).
//
// Warps (384 threads): 0 TMA producer, 1 tensor-memory owner and (leader CTA) MMA
// issuer, 2-3 idle, 4-11 epilogue.  Two accumulators let the epilogue of one tile
// overlap the main loop of the next.  The persistent schedule walks tiles in groups
// of 8 m-tiles; a last round that would fill at most half of the CTA pairs runs its
// tiles as two column halves (at BN = 256).
#pragma once

#include "ffn_act.cuh"
#include "ffn_ptx.cuh"
#include "gemm_tc.cuh"

namespace igc {

enum class FfnOp : int { Linear = 0, Gated = 1, GradX = 2, GradW = 3 };

__host__ __device__ constexpr bool ffn_a_mn(FfnOp o) { return o == FfnOp::GradW; }
__host__ __device__ constexpr bool ffn_b_mn(FfnOp o) {
  return o == FfnOp::GradX || o == FfnOp::GradW;
}

constexpr int kFfnThreads = 128 + 32 * kEpiWarps;  // 384
constexpr int kFfnAtoms = 2;                       // 128-deep stages
constexpr int kFfnKS = BK * kFfnAtoms;
constexpr int kFfnBox = 64;  // columns of one epilogue box (128 bytes of a 16-bit output)

// Least dynamic shared memory of a CTA that allocates `cols` columns of tensor memory.  An
// SM has 512 of them, an allocation waits without limit for too few, and CTAs of any launch,
// those of other streams among them, may share the SM.  So shared memory is asked for in
// proportion: columns come in 32s, CTAs that together want more than 512 want 544 at least,
// and 544 columns' worth is the whole of an SM's 228 KB, without what a CTA needs besides.
constexpr size_t kSmemPerSm = 228 * 1024;
constexpr size_t tmem_smem_floor(uint32_t cols) { return (kSmemPerSm * cols + 543) / 544; }

template <FfnOp kOp, int BN>
struct FfnCfg {
  static constexpr int kOutN = kOp == FfnOp::Gated ? BN / 2 : BN;  // output columns of a tile
  static_assert(BN % 64 == 0 && BN <= 256 && kOutN % kFfnBox == 0, "BN");
  static constexpr uint32_t kStageA = kAtomABytes * kFfnAtoms;
  // MN-major atoms hold a CTA's BN/2 rows of B in groups of 64
  static_assert(!ffn_b_mn(kOp) || BN % 128 == 0, "BN");
  static constexpr uint32_t kAtomB = BN / 2 * BK * 2;
  static constexpr uint32_t kStageB = kAtomB * kFfnAtoms;
  static constexpr uint32_t kStageBytes = kStageA + kStageB;
  static constexpr int kStages =
      static_cast<int>((kSmemBudget - 2048 - kStagingBytes) / kStageBytes) > 8
          ? 8
          : static_cast<int>((kSmemBudget - 2048 - kStagingBytes) / kStageBytes);
  static constexpr uint32_t kAccStride = BN <= 128 ? 128 : 256;  // columns of an accumulator
  static constexpr uint32_t kTmemCols = 2 * kAccStride;
  static constexpr size_t kSmemUsed = 1024 + kStages * kStageBytes + kStagingBytes + 1024;
  static constexpr size_t kSmemBytes =
      kSmemUsed > tmem_smem_floor(kTmemCols) ? kSmemUsed : tmem_smem_floor(kTmemCols);
  static_assert(kSmemBytes <= kSmemBudget, "shared memory");
  static constexpr bool kHalves = BN == 256;  // column-half units in the last round
};

// One output matrix of the epilogue.
struct FfnOut {
  void* ptr;
  long long ld;
  int f32;    // fp32 elements, else 16-bit
  int tma;    // written by bulk tensor stores
  int whole;  // rows of whole 16-byte pieces
};

struct FfnParams {
  int M, N;      // rows and columns of one output matrix
  int kb_seg;    // pipeline stages of one contraction segment
  int segs;      // contraction segments (GradX: pairs of operands summed)
  int srcs;      // output matrices stacked along m (GradW)
  int tiles_m;   // m-tiles of one output matrix
  int tiles_n, num_tiles, group_m, tail_start, num_units;
  int bf16;      // operand type (else fp16)
  int late_wait; // see ffn_dependency_wait
  int act;
  const void* bias0;
  const void* bias1;
  int bias_f32;
  const void* R;
  long long ldr;
  int r_vec;
  // Linear: 0 = Y, 1 = Z; Gated: 0 = H, 1 = G, 2 = U; GradX: 0 = dX; GradW: s = dW_s
  FfnOut out[3];
  unsigned long long wait_limit_ns;
  unsigned long long* status;
};

// Programmatic dependent launch.  A kernel normally waits for the one before it in the
// stream before it touches memory.  With `late` it may run beside it: they share no memory
// that either of them writes, and what it does read is complete when it starts.  In a
// backward pass A, B, C, D (the activation's pass, dX, dW, the bias sums) C and D are late
// and read what A wrote.  B waits for A and lets C start only then, from every block; so C
// starts after A's end, and D, which C's blocks let start, after that.  Both pass over A's
// results in L2 (TMA, __ldcg), which is where a finished kernel's stores are.  A late kernel
// waits for the one before it at its end: D's end means C's, C's means B's, so whatever
// follows D in the stream finds all of them complete.
__device__ __forceinline__ void ffn_dependency_wait(bool late) {
  if (!late) grid_dependency_wait();
  grid_dependents_launch();
}
__device__ __forceinline__ void ffn_dependency_end(bool late) {
  if (late) grid_dependency_wait();
}

// A unit of the schedule: the columns [n0, n0 + cols) of m-tile mb.
struct FfnUnit {
  int mb, n0, cols, half;
};

template <FfnOp kOp, int BN>
__device__ __forceinline__ FfnUnit ffn_unit(const FfnParams& p, int u) {
  constexpr int kOutN = FfnCfg<kOp, BN>::kOutN;
  int t = u, j = 0, half = 0;
  if (u >= p.tail_start) {
    t = p.tail_start + ((u - p.tail_start) >> 1);
    j = (u - p.tail_start) & 1;
    half = 1;
  }
  const int tm = p.tiles_m * p.srcs;
  const int per_group = p.group_m * p.tiles_n;
  const int g = t / per_group;
  const int first_m = g * p.group_m;
  const int gm = min(tm - first_m, p.group_m);
  const int r = t - g * per_group;
  FfnUnit w;
  w.mb = first_m + r % gm;
  w.cols = half ? kOutN / 2 : kOutN;
  w.n0 = (r / gm) * kOutN + j * w.cols;
  w.half = half;
  return w;
}

// One stage's copies of one CTA.  ka: k of the stage within its segment.
template <FfnOp kOp, int BN>
__device__ __forceinline__ void ffn_load_stage(const CUtensorMap* tmA, const CUtensorMap* tmB,
                                               uint8_t* a_dst, uint8_t* b_dst, uint32_t bar,
                                               int ka, int m_cta, int n_cta, int half) {
  using Cfg = FfnCfg<kOp, BN>;
  constexpr uint32_t kMnGroup = 64 * 2 * kFfnKS;  // bytes of 64 outputs x one stage of k
  if constexpr (ffn_a_mn(kOp)) {
#pragma unroll
    for (int g = 0; g < BM_CTA / 64; ++g)
      tma_load_2d_2cta(a_dst + g * kMnGroup, tmA, bar, m_cta + 64 * g, ka);
  } else {
#pragma unroll
    for (int j = 0; j < kFfnAtoms; ++j)
      tma_load_2d_2cta(a_dst + j * kAtomABytes, tmA, bar, ka + j * BK, m_cta);
  }
  if constexpr (ffn_b_mn(kOp)) {
#pragma unroll
    for (int g = 0; g < BN / 2 / 64; ++g)
      if (g == 0 || !half) tma_load_2d_2cta(b_dst + g * kMnGroup, tmB, bar, n_cta + 64 * g, ka);
  } else {
    // boxes of BN/4 rows: one for a half unit, two for a whole one
#pragma unroll
    for (int j = 0; j < kFfnAtoms; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (q == 0 || !half)
          tma_load_2d_2cta(b_dst + j * Cfg::kAtomB + q * (BN / 4) * 128, tmB, bar, ka + j * BK,
                           n_cta + q * (BN / 4));
  }
}

// One stage's MMAs: kFfnKS / 16 steps of k = 16.
template <FfnOp kOp, int BN>
__device__ __forceinline__ void ffn_mma_stage(uint32_t d_tmem, uint64_t a_st, uint64_t b_st,
                                              uint32_t idesc, bool accumulate) {
  using Cfg = FfnCfg<kOp, BN>;
#pragma unroll
  for (int i = 0; i < kFfnKS / 16; ++i) {
    // MN-major: 16 k are two 8-k groups (2048 bytes); K-major: 32 bytes of a row
    const uint32_t a_off = ffn_a_mn(kOp) ? i * 2048u : (i / 4) * kAtomABytes + (i % 4) * 32u;
    const uint32_t b_off = ffn_b_mn(kOp) ? i * 2048u : (i / 4) * Cfg::kAtomB + (i % 4) * 32u;
    umma_f16_ss_2cta(d_tmem, a_st + (a_off >> 4), b_st + (b_off >> 4), idesc,
                     (accumulate || i > 0) ? 1u : 0u);
  }
}

// ---------------------------------------------------------------------------
// epilogue: a warp owns 32 rows (a row per lane) and one box of 64 columns at a time
// ---------------------------------------------------------------------------

// Byte offset, in a warp's staging buffer, of 16-bit element c of row r (Stager::put's layout).
__device__ __forceinline__ int ffn_staged(int r, int c) {
  return r * 128 + ((((c >> 3) ^ (r & 7)) << 4) | ((c & 7) << 1));
}

// Stores a box that TMA cannot store, from the staging buffer: a row at a time, a column
// per lane, so that a warp's stores fall into the few sectors of one row.  kWords: fp32 (32
// columns), else 16-bit (64 columns).
template <bool kWords>
__device__ __forceinline__ void ffn_store_rows(const FfnOut& o, const Stager& st, int n0) {
  __syncwarp();
  const int rows = min(32, st.M - st.row0);
  for (int r = 0; r < rows; ++r) {
    const long long at = static_cast<long long>(st.row0 + r) * o.ld + n0;
    if constexpr (kWords) {
      if (n0 + st.lane < st.N)
        static_cast<float*>(o.ptr)[at + st.lane] =
            *reinterpret_cast<const float*>(st.buf + ffn_staged(r, 2 * st.lane));
    } else {
#pragma unroll
      for (int c = st.lane; c < kFfnBox; c += 32)
        if (n0 + c < st.N)
          static_cast<uint16_t*>(o.ptr)[at + c] =
              *reinterpret_cast<const uint16_t*>(st.buf + ffn_staged(r, c));
    }
  }
  __syncwarp();
}

// Stores one box: the 128 bytes of this lane's row (64 16-bit or 32 fp32 columns from n0).
// TMA leaves out what lies past the last column in pieces of 16 bytes only: a box with a
// broken last piece would be written past the matrix, so it goes row by row.
template <bool kWords>
__device__ __forceinline__ void ffn_store_box(const FfnOut& o, const CUtensorMap* map,
                                              const Stager& st, int n0, const uint32_t (&v)[32]) {
  st.begin();
#pragma unroll
  for (int k = 0; k < 8; ++k)
    st.put(k, make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]));
  if (o.tma && (o.whole || n0 + (kWords ? kFfnBox / 2 : kFfnBox) <= st.N))
    st.issue(map, n0);
  else
    ffn_store_rows<kWords>(o, st, n0);
}

// What a box's epilogue reads besides the accumulator, fetched before the accumulator is
// waited for: the biases of columns n0 + lane and n0 + 32 + lane (broadcast by shuffles
// later) and this lane's row of the residual.
struct FfnFetched {
  float bias0[2], bias1[2];
  uint4 res[8];
};

// The residual's box where rows are not 16-byte aligned: a row at a time through the
// staging buffer, a column per lane.
__device__ __forceinline__ void ffn_gather_residual(const FfnParams& p, const Stager& st, int n0,
                                                    FfnFetched& f) {
  st.begin();
  const uint16_t* src = static_cast<const uint16_t*>(p.R);
  const int rows = min(32, st.M - st.row0);
  for (int r0 = 0; r0 < rows; r0 += 16) {
    uint16_t e[16][2];
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int n = n0 + st.lane + 32 * h;
        e[j][h] = r0 + j < rows && n < p.N
                      ? src[static_cast<long long>(st.row0 + r0 + j) * p.ldr + n]
                      : static_cast<uint16_t>(0);
      }
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<uint16_t*>(st.buf + ffn_staged(r0 + j, st.lane + 32 * h)) = e[j][h];
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k)
    f.res[k] = *reinterpret_cast<const uint4*>(st.buf + ffn_staged(st.lane, 8 * k));
  __syncwarp();
}

template <FfnOp kOp>
__device__ __forceinline__ void ffn_fetch(const FfnParams& p, const Stager& st, int n0,
                                          FfnFetched& f) {
  if constexpr (kOp == FfnOp::Linear || kOp == FfnOp::Gated) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int n = n0 + 32 * c + st.lane;
      f.bias0[c] = n < p.N ? load_vec(p.bias0, n, p.bias_f32, p.bf16) : 0.0f;
      if constexpr (kOp == FfnOp::Gated)
        f.bias1[c] = n < p.N ? load_vec(p.bias1, n, p.bias_f32, p.bf16) : 0.0f;
    }
  }
  if constexpr (kOp == FfnOp::Linear) {
    if (p.R == nullptr) return;
    if (p.r_vec) {
      const int m = st.row0 + st.lane;
      const int cols = m < p.M ? p.N - n0 : 0;
      const uint16_t* r =
          static_cast<const uint16_t*>(p.R) + static_cast<long long>(m) * p.ldr + n0;
      if (cols >= kFfnBox) {
#pragma unroll
        for (int k = 0; k < 8; ++k) f.res[k] = reinterpret_cast<const uint4*>(r)[k];
      } else {
        // 16 bytes at a time, the row's last columns, where they do not fill 16, singly
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t w[4] = {0u, 0u, 0u, 0u};
          if (8 * k + 8 <= cols) {
            const uint4 q = reinterpret_cast<const uint4*>(r)[k];
            w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
          } else if (8 * k < cols) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (8 * k + i < cols)
                w[i / 2] |= static_cast<uint32_t>(r[8 * k + i]) << (16 * (i & 1));
          }
          f.res[k] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    } else {
      ffn_gather_residual(p, st, n0, f);
    }
  }
}

__device__ __forceinline__ void ffn_add_bias(float b, float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] += __shfl_sync(0xffffffffu, b, i);
}

// v += the residual's columns n0 + 32 c .. + 31.
__device__ __forceinline__ void ffn_add_residual(const FfnParams& p, const FfnFetched& f, int c,
                                                 float (&v)[32]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint4 q = f.res[4 * c + k];
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 e = unpack16(w[i], p.bf16);
      v[8 * k + 2 * i] += e.x;
      v[8 * k + 2 * i + 1] += e.y;
    }
  }
}

__device__ __forceinline__ void ffn_pack(const float (&v)[32], uint32_t* dst, bool bf16) {
#pragma unroll
  for (int i = 0; i < 16; ++i) dst[i] = pack16(v[2 * i], v[2 * i + 1], bf16);
}

__device__ __forceinline__ void ffn_tmem_load(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  tmem_ld_32x32b_x32(taddr, r);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// One box (64 columns from n0) of this warp's rows.  acc: tensor-memory address of
// the box's first column; for Gated, U lies u_off columns further.
template <FfnOp kOp>
__device__ __forceinline__ void ffn_epilogue_box(const FfnParams& p, const CUtensorMap* tmO0,
                                                 const CUtensorMap* tmO1, const CUtensorMap* tmO2,
                                                 const Stager& st, uint32_t acc, int u_off,
                                                 const FfnFetched& f, int n0, int src) {
  const bool bf16 = p.bf16 != 0;
  if constexpr (kOp == FfnOp::Gated) {
    uint32_t h[32], gk[32], uk[32];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float g[32], u[32];
      ffn_tmem_load(acc + 32 * c, g);
      ffn_tmem_load(acc + u_off + 32 * c, u);
      if (p.bias0 != nullptr) ffn_add_bias(f.bias0[c], g);
      if (p.bias1 != nullptr) ffn_add_bias(f.bias1[c], u);
      if (p.out[1].ptr != nullptr) {
        ffn_pack(g, gk + 16 * c, bf16);
        ffn_pack(u, uk + 16 * c, bf16);
      }
      with_act(p.act, [&](auto a) {
#pragma unroll
        for (int i = 0; i < 32; ++i) g[i] = act_f32<decltype(a)::value>(g[i]) * u[i];
      });
      ffn_pack(g, h + 16 * c, bf16);
    }
    ffn_store_box<false>(p.out[0], tmO0, st, n0, h);
    if (p.out[1].ptr != nullptr) {
      ffn_store_box<false>(p.out[1], tmO1, st, n0, gk);
      ffn_store_box<false>(p.out[2], tmO2, st, n0, uk);
    }
  } else {
    // GradW's second matrix is written through slot 1
    const FfnOut& o = (kOp == FfnOp::GradW && src) ? p.out[1] : p.out[0];
    const CUtensorMap* map = (kOp == FfnOp::GradW && src) ? tmO1 : tmO0;
    uint32_t y[32], z[32];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int n = n0 + 32 * c;
      float v[32];
      ffn_tmem_load(acc + 32 * c, v);
      if constexpr (kOp == FfnOp::Linear) {
        if (p.bias0 != nullptr) ffn_add_bias(f.bias0[c], v);
        if (p.out[1].ptr != nullptr) ffn_pack(v, z + 16 * c, bf16);
        with_act(p.act, [&](auto a) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = act_f32<decltype(a)::value>(v[i]);
        });
        if (p.R != nullptr) ffn_add_residual(p, f, c, v);
      }
      if (o.f32) {
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(v[i]);
        if (n < p.N) ffn_store_box<true>(o, map, st, n, w);
      } else {
        ffn_pack(v, y + 16 * c, bf16);
      }
    }
    if (!o.f32) ffn_store_box<false>(o, map, st, n0, y);
    if constexpr (kOp == FfnOp::Linear)
      if (p.out[1].ptr != nullptr) ffn_store_box<false>(p.out[1], tmO1, st, n0, z);
  }
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <FfnOp kOp, int BN>
__global__ void __launch_bounds__(kFfnThreads, 1)
    igc_ffn_gemm_kernel(const __grid_constant__ CUtensorMap tmA0,
                        const __grid_constant__ CUtensorMap tmA1,
                        const __grid_constant__ CUtensorMap tmB0,
                        const __grid_constant__ CUtensorMap tmB1,
                        const __grid_constant__ CUtensorMap tmO0,
                        const __grid_constant__ CUtensorMap tmO1,
                        const __grid_constant__ CUtensorMap tmO2, const FfnParams p) {
  using Cfg = FfnCfg<kOp, BN>;
  constexpr int kStages = Cfg::kStages;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sA = smem;
  uint8_t* sB = smem + kStages * Cfg::kStageA;
  uint8_t* staging = sB + kStages * Cfg::kStageB;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kStagingBytes);  // leader's are used
  uint64_t* empty = full + kStages;   // each CTA: stage s may be overwritten
  uint64_t* tfull = empty + kStages;  // each CTA: accumulator a is ready
  uint64_t* tempty = tfull + 2;       // leader: both epilogues released accumulator a
  uint64_t* mma_done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 32, 0);
  const int lane = static_cast<int>(lane_id());
  const uint32_t rank = cluster_ctarank();  // 0 = leader
  const int cluster = static_cast<int>(blockIdx.x) >> 1;
  const int num_clusters = static_cast<int>(gridDim.x) >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * kEpiWarps);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA0);
    tma_prefetch_desc(&tmB0);
  }
  if (warp == 1) {
    tmem_alloc_2cta(tmem_slot, Cfg::kTmemCols);
    tmem_relinquish_2cta();
  }
  tc_fence_before();
  cluster_sync();  // barriers of both CTAs initialised, tensor memory allocated in both
  tc_fence_after();
  // nothing above touches global memory; from here on the previous kernel in the
  // stream must have finished (programmatic dependent launch)
  ffn_dependency_wait(p.late_wait);
  const uint32_t tmem_base = *tmem_slot;
  const uint64_t lim = p.wait_limit_ns;
  // the pair's MMAs write both CTAs' tensor memory at the leader's address
  const bool pair_ok =
      ld_shared_cluster_u32(mapa_shared(smem_u32(tmem_slot), rank ^ 1u)) == tmem_base;
  if (!pair_ok && threadIdx.x == 0) report_status(p.status, kStatusBadLaunch, kSiteTmemMismatch);
  const uint32_t full_lead = mapa_shared(smem_u32(full), 0);
  const uint32_t tempty_lead = mapa_shared(smem_u32(tempty), 0);

  if (pair_ok && warp == 0) {
    // ---------------------------------------------------------------- producer
    int stage = 0;
    uint32_t phase = 0;
    long long issued = 0;
    for (int u = cluster; u < p.num_units; u += num_clusters) {
      const FfnUnit w = ffn_unit<kOp, BN>(p, u);
      const int src = kOp == FfnOp::GradW ? w.mb / p.tiles_m : 0;
      const int m_cta = (w.mb - src * p.tiles_m) * BM + static_cast<int>(rank) * BM_CTA;
      const int n_cta =
          kOp == FfnOp::Gated ? w.n0 : w.n0 + static_cast<int>(rank) * (w.cols / 2);
      const uint32_t stage_tx =
          2u * (Cfg::kStageA + (w.half ? Cfg::kStageB / 2 : Cfg::kStageB));
      for (int seg = 0; seg < p.segs; ++seg) {
        const CUtensorMap* mapA = (kOp == FfnOp::GradX ? seg : src) ? &tmA1 : &tmA0;
        const bool b1 = kOp == FfnOp::GradX ? seg != 0 : (kOp == FfnOp::Gated && rank != 0);
        const CUtensorMap* mapB = b1 ? &tmB1 : &tmB0;
        for (int kb = 0; kb < p.kb_seg; ++kb) {
          if (!__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1u, lim, abort_flag,
                                                  p.status, kSiteProducerEmpty)))
            goto producer_done;
          if (lane == 0) {
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], stage_tx);
            ffn_load_stage<kOp, BN>(mapA, mapB, sA + stage * Cfg::kStageA,
                                    sB + stage * Cfg::kStageB,
                                    full_lead + static_cast<uint32_t>(stage) * 8u, kb * kFfnKS,
                                    m_cta, n_cta, w.half);
          }
          __syncwarp();
          ++issued;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
  producer_done:
    if (lane == 0 && *abort_flag && issued > 0) {
      // The copies signal the leader's barriers; this CTA's own copies in flight get
      // time to land before the CTA may exit (a copy takes microseconds).
      if (rank == 0) {
        drain_fills(full, kStages, stage, phase, issued, lim);
      } else {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000ull) {
        }
      }
    }
  } else if (pair_ok && warp == 1 && rank == 0) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t kMajor =
        (ffn_a_mn(kOp) ? 1u << 15 : 0u) | (ffn_b_mn(kOp) ? 1u << 16 : 0u);
    const uint32_t fmt = p.bf16 ? 1u : 0u;
    const uint32_t idesc_full = make_idesc_kind_f16(BM, BN, fmt) | kMajor;
    const uint32_t idesc_half = make_idesc_kind_f16(BM, BN / 2, fmt) | kMajor;
    constexpr uint32_t kMnGroup = 64 * 2 * kFfnKS;
    const uint64_t adesc0 = ffn_a_mn(kOp) ? make_sw128_mnmajor_desc(smem_u32(sA), kMnGroup)
                                          : make_sw128_kmajor_desc(smem_u32(sA));
    const uint64_t bdesc0 = ffn_b_mn(kOp) ? make_sw128_mnmajor_desc(smem_u32(sB), kMnGroup)
                                          : make_sw128_kmajor_desc(smem_u32(sB));
    const int num_kb = p.kb_seg * p.segs;
    int stage = 0;
    uint32_t phase = 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int u = cluster; u < p.num_units; u += num_clusters) {
      const uint32_t idesc = u >= p.tail_start ? idesc_half : idesc_full;
      if (!__all_sync(0xffffffffu, mbar_wait(&tempty[acc], acc_phase ^ 1u, lim, abort_flag,
                                              p.status, kSiteMmaTmemEmpty)))
        goto mma_done_label;
      tc_fence_after();
      for (int kb = 0; kb < num_kb; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], phase, lim, abort_flag, p.status,
                                                kSiteMmaFull)))
          goto mma_done_label;
        tc_fence_after();
        if (lane == 0) {
          ffn_mma_stage<kOp, BN>(
              tmem_base + static_cast<uint32_t>(acc) * Cfg::kAccStride,
              adesc0 + ((static_cast<uint32_t>(stage) * Cfg::kStageA) >> 4),
              bdesc0 + ((static_cast<uint32_t>(stage) * Cfg::kStageB) >> 4), idesc, kb > 0);
          umma_commit_2cta_multicast(&empty[stage], 0x3);
          if (kb == num_kb - 1) umma_commit_2cta_multicast(&tfull[acc], 0x3);
        }
        __syncwarp();
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  mma_done_label:
    if (lane == 0) {
      // every MMA issued by this thread has finished once mma_done completes
      umma_commit_2cta(mma_done);
      int dummy = 0;
      mbar_wait(mma_done, 0, lim, &dummy, p.status, kSiteDrain);
    }
    __syncwarp();
  } else if (pair_ok && warp >= 4) {
    // ---------------------------------------------------------------- epilogue
    const int ew = warp - 4;
    const int quad = warp & 3;  // tcgen05.ld: warp w may access lanes 32 (w % 4) .. +31
    const int first_box = ew >> 2;
    Stager st;
    st.buf = staging + ew * kStagingWarpBytes;
    st.lane = lane;
    st.M = p.M;
    st.N = p.N;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int u = cluster; u < p.num_units; u += num_clusters) {
      const FfnUnit w = ffn_unit<kOp, BN>(p, u);
      const int src = kOp == FfnOp::GradW ? w.mb / p.tiles_m : 0;
      st.row0 = (w.mb - src * p.tiles_m) * BM + static_cast<int>(rank) * BM_CTA + quad * 32;
      FfnFetched f;
      ffn_fetch<kOp>(p, st, w.n0 + first_box * kFfnBox, f);
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[acc], acc_phase, lim, abort_flag, p.status,
                                              kSiteEpiFull)))
        goto epi_done;
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) +
                             static_cast<uint32_t>(acc) * Cfg::kAccStride;
      for (int b = first_box; b < w.cols / kFfnBox && w.n0 + b * kFfnBox < p.N; b += 2) {
        if (b != first_box) ffn_fetch<kOp>(p, st, w.n0 + b * kFfnBox, f);
        ffn_epilogue_box<kOp>(p, &tmO0, &tmO1, &tmO2, st,
                              taddr + static_cast<uint32_t>(b * kFfnBox), w.cols, f,
                              w.n0 + b * kFfnBox, src);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(tempty_lead + static_cast<uint32_t>(acc) * 8u);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  epi_done:
    // every staged store of this warp has completed before the CTA may exit
    if (lane == 0) bulk_wait_group0();
    __syncwarp();
  }

  // ------------------------------------------------------------------ teardown
  // No CTA of the pair may exit (or free tensor memory) while its peer can still
  // touch its shared memory or barriers.
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_2cta(tmem_base, Cfg::kTmemCols);
  }
  ffn_dependency_end(p.late_wait);
}

}  // namespace igc
