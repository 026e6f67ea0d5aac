// Backward pass of layer norm: the kernels and their launch for one type of dY and dX (kT) and
// one of S, A and dS (kS).
//
//   h = (S - mean) rstd      g = dY w
//   dS = rstd (g - mean of g - h mean of g h) + A       dX = drop(dS)
//   dw = column sums of dY h                            db = column sums of dY
//
// Bound by memory: dY, S and A are read once, dS and dX written once.  A fixed number of blocks
// walks down the rows: the column sums of a thread's columns stay in its registers over all of
// them, one row of partial sums per block goes to the workspace, and a second kernel adds the
// blocks' in order (no atomics).  16384 x 4096 bf16 with dropout and A: 106 us, 671 MB at 6.3 TB/s.
#pragma once

#include "row_stream_host.h"

namespace igc {

struct NormBwdParams {
  int M, N, vec, w_f32;
  const void* dY;
  const void* S;
  const void* A;
  void* dS;
  void* dX;
  long long lddy, lds, lda, ldds, lddx;
  const float* mean;
  const float* rstd;
  const void* w;
  float* partial;  // [2][blocks][N]: dw, db (null: no column sums)
  void* dw;        // written by the cluster that all blocks are, if they are one (join)
  void* db;
  int join, dw_f32;
  Drop drop;
};

// A batch of few rows is taken by at most this many blocks, one cluster: it adds the blocks' sums
// through distributed shared memory and writes dw and db itself, one launch less.
constexpr int kJoinBlocks = 8;

constexpr int kMaxPartials = 512;  // rows of partial sums that the workspace has room for

// dS of eight columns from g, h and the row's sums.
template <int kS>
__device__ __forceinline__ void slopes8(const NormBwdParams& p, float rstd, float c1, float c2,
                                        const Raw8<kS>& a, const float (&g)[8],
                                        const float (&h)[8], float (&d)[8]) {
  float f[8] = {};
  if (p.A != nullptr) unpack8<kS>(a, f);
  const uint64_t r = pair(rstd, rstd), m1 = pair(-c1, -c1), m2 = pair(-c2, -c2);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const uint64_t x = fma2(pair(h[j], h[j + 1]), m2, add2(pair(g[j], g[j + 1]), m1));
    unpair(fma2(x, r, pair(f[j], f[j + 1])), d[j], d[j + 1]);
  }
}

// The sums of one column by `blocks` blocks of a cluster, in order, where each has them at `sums`
// (in its own shared memory).
__device__ __forceinline__ float cluster_sum(const float* sums, int blocks) {
  float total = 0.0f;
#pragma unroll
  for (int r = 0; r < kJoinBlocks; ++r)
    if (r < blocks)
      total += __uint_as_float(
          ld_shared_cluster_u32(mapa_shared(smem_u32(sums), static_cast<uint32_t>(r))));
  return total;
}

// The whole cluster: dw and db from the blocks' sums dw_sums[n] and db_sums[n], columns dealt
// over the blocks.
template <int kT>
__device__ __noinline__ void join_sums(const NormBwdParams& p, const float* dw_sums,
                                          const float* db_sums) {
  const int blocks = static_cast<int>(gridDim.x);
  cluster_sync();
  for (int n = static_cast<int>(blockIdx.x * blockDim.x + threadIdx.x); n < p.N;
       n += blocks * static_cast<int>(blockDim.x)) {
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      void* out = v ? p.db : p.dw;
      if (out == nullptr) continue;
      const float sum = cluster_sum((v ? db_sums : dw_sums) + n, blocks);
      if (kT == IGC_F32 || p.dw_f32)
        static_cast<float*>(out)[n] = sum;
      else
        store16(out, n, sum, kT == IGC_BF16);
    }
  }
  cluster_sync();  // no block may exit while another reads its sums
}

// g and h of eight columns from dY (g) and S (h), with their part of the row's sums and of the
// column sums.  Past the row's end dY is 0 and S the mean: a 0 of S there would make h infinite
// where the mean is far from 0, and its product with g = 0 NaN.
template <bool kSums>
__device__ __forceinline__ void terms8(float mean, float rstd, const float (&w)[8], float (&g)[8],
                                       float (&h)[8], uint64_t& c1, uint64_t& c2, float (&sw)[8],
                                       float (&sb)[8]) {
  const uint64_t m = pair(-mean, -mean), r = pair(rstd, rstd);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const uint64_t hh = mul2(add2(pair(h[j], h[j + 1]), m), r);
    const uint64_t y = pair(g[j], g[j + 1]);
    if constexpr (kSums) {
      unpair(fma2(y, hh, pair(sw[j], sw[j + 1])), sw[j], sw[j + 1]);
      unpair(add2(y, pair(sb[j], sb[j + 1])), sb[j], sb[j + 1]);
    }
    const uint64_t gg = mul2(y, pair(w[j], w[j + 1]));
    c1 = add2(c1, gg);
    c2 = fma2(gg, hh, c2);
    unpair(gg, g[j], g[j + 1]);
    unpair(hh, h[j], h[j + 1]);
  }
}

constexpr int kNormBwdStreamMost = 512;  // 128 registers each

// Rows streamed through shared memory (row_stream.cuh), two or three units to a thread (three:
// dY and S are taken from the slot again after the sums, their registers go to the column sums).
// Rows of more columns than a block has are shared by the kCluster blocks of a cluster, which
// exchange their sums through distributed shared memory.
template <int kT, int kS, int kLanes, int kUnits, int kCluster, bool kDrop>
__global__ void __launch_bounds__(stream_threads(kLanes, kNormBwdStreamMost), 1)
    layer_norm_bwd_stream_kernel(const NormBwdParams p, const RowStream st) {
  constexpr int kGroups = kNormBwdStreamMost / kLanes;
  constexpr bool kAgain = kUnits > 2;  // g and h are formed again after the sums
  constexpr int kSizeT = kT == IGC_F32 ? 4 : 2, kSizeS = kS == IGC_F32 ? 4 : 2;
  extern __shared__ __align__(128) char ring[];
  __shared__ uint64_t full[kGroups][kMaxSlots];
  __shared__ __align__(16) float2 red[kGroups][2][(kLanes / 32 + 1) / 2 * 2];
  __shared__ __align__(16) Meeting<kCluster> meet[kCluster > 1 ? kGroups : 1];
  __shared__ int abort_flag, lost;
  const RowWalk walk =
      row_walk<kLanes, kGroups, kCluster>(st, ring, full, &abort_flag, &lost, p.M);
  if constexpr (kCluster > 1) {
    if (walk.t == 0) {
      Meeting<kCluster>& m = meet[walk.group];
      mbar_init(&m.bar[0], 1);
      mbar_init(&m.bar[1], 1);
      fence_mbar_init();
#pragma unroll
      for (int r = 0; r < kCluster; ++r) m.sent[r] = walk.count;
    }
    cluster_sync();
  }
  grid_dependency_wait();
  grid_dependents_launch();
  // this block's columns [col0, col0 + cols), whole units
  const int t = walk.t, N8 = p.N / 8 * 8, share = (N8 / 8 + kCluster - 1) / kCluster * 8;
  const int rank = kCluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int col0 = rank * share, cols = min(share, N8 - col0);
  const bool has_a = p.A != nullptr, has_s = p.dS != nullptr, has_x = p.dX != nullptr;
  auto fill = [&](int k) {
    const long long row = walk.first + k * walk.step;
    const int slot = k % st.slots;
    const char* const from[kStreamMats] = {row_at<kT>(p.dY, row, p.lddy) + col0 * kSizeT,
                                           row_at<kS>(p.S, row, p.lds) + col0 * kSizeS,
                                           row_at<kS>(p.A, row, p.lda) + col0 * kSizeS};
    fill_slot(st, walk.slots + slot * st.slot_bytes, walk.bars + slot, from,
              static_cast<uint32_t>(cols));
  };
  // A group of one warp refills a slot when its row is done; a larger one after the barrier of
  // the next row, a row later: it fills one slot less at first.
  constexpr int kBehind = kLanes == 32 ? 0 : 1;
  if (t == 0)
    for (int k = 0; k < walk.count && k < st.slots - kBehind; ++k) fill(k);
  keep_weights<kT>(ring, st.plane, p.w, col0, cols, p.w_f32);
  __syncthreads();
  const uint64_t offset = kDrop ? drop_offset(p.drop) : 0;
  const float inv = 1.0f / static_cast<float>(p.N);
  float sw[kUnits][8] = {}, sb[kUnits][8] = {}, sw_last = 0.0f, sb_last = 0.0f;
  // the column past the whole units that this thread has, if any; the next row's statistics and
  // its elements there arrive during a row
  const int last = rank == kCluster - 1 && N8 + t < p.N ? N8 + t : -1;
  const float w_last =
      last >= 0 && p.w != nullptr
          ? load_vec(p.w, last, kT == IGC_F32 || p.w_f32, kT == IGC_BF16)
          : 1.0f;
  float mean = 0.0f, rstd = 0.0f, y_last = 0.0f, s_last = 0.0f, a_last = 0.0f;
  auto load_last = [&](long long row) {
    y_last = load1<kT>(row_at<kT>(p.dY, row, p.lddy), last);
    s_last = load1<kS>(row_at<kS>(p.S, row, p.lds), last);
    if (has_a) a_last = load1<kS>(row_at<kS>(p.A, row, p.lda), last);
  };
  if (walk.count > 0) {
    mean = p.mean[walk.first], rstd = p.rstd[walk.first];
    if (last >= 0) load_last(walk.first);
  }
  char* ds_row = row_at<kS>(p.dS, walk.first, p.ldds) + col0 * kSizeS;
  char* dx_row = row_at<kT>(p.dX, walk.first, p.lddx) + col0 * kSizeT;
  const long long ds_step = walk.step * p.ldds * kSizeS, dx_step = walk.step * p.lddx * kSizeT;
  // A wait that gave up is reported; the group goes on to its end, without further copies, waits
  // and sums sent.
  int stop = -1;  // twice the row whose wait gave up, plus 1 where that was for the cluster's sums
  int slot = 0;
  uint32_t phase = 0;
  // whole: every lane of the warp has all its units, so that no branch keeps the loads and the
  // arithmetic of different units apart (16384 x 4096 bf16 with dropout: 106 us, with a branch
  // for each unit 119)
  auto walk_rows = [&](auto whole) {
    for (int k = 0; k < walk.count; ++k) {
      const long long row = walk.first + k * walk.step;
      const char* at = walk.slots + slot * st.slot_bytes;
      float mean_next = 0.0f, rstd_next = 0.0f;
      if (k + 1 < walk.count)
        mean_next = p.mean[row + walk.step], rstd_next = p.rstd[row + walk.step];
      if (!mbar_try_wait(smem_u32(walk.bars + slot), phase) && stop < 0 &&
          !mbar_wait(walk.bars + slot, phase, st.wait_limit, &abort_flag, st.status,
                     kSiteNormBwdRow))
        stop = 2 * k;
      float g[kAgain ? 1 : kUnits][8], h[kAgain ? 1 : kUnits][8];
      uint64_t p1 = 0, p2 = 0;
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int n = (i * kLanes + t) * 8, q = kAgain ? 0 : i;
        if (!decltype(whole)::value && n >= cols) continue;
        float wv[8];
        kept_weights(ring, st.plane, n, wv);
        load_unit<kT>(at + st.at[0] + n * kSizeT, g[q]);
        load_unit<kS>(at + st.at[1] + n * kSizeS, h[q]);
        terms8<true>(mean, rstd, wv, g[q], h[q], p1, p2, sw[i], sb[i]);
      }
      float c1 = sum2(p1), c2 = sum2(p2), g_last = 0.0f, h_last = 0.0f, f_last = a_last;
      if (last >= 0) {
        h_last = (s_last - mean) * rstd;
        sw_last = fmaf(y_last, h_last, sw_last);
        sb_last += y_last;
        g_last = y_last * w_last;
        c1 += g_last;
        c2 = fmaf(g_last, h_last, c2);
        if (k + 1 < walk.count) load_last(row + walk.step);
      }
      // the bits of the dropout are made here, among the shuffles of the sums
      [[maybe_unused]] uint4 bits[kDrop && !kAgain ? kUnits : 1];
      if constexpr (kDrop && !kAgain) {
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
          bits[i] = drop_bits(p.drop, offset, row, col0 + (i * kLanes + t) * 8);
      }
      if constexpr (kLanes == 32) {
        lane_sums<32>(c1, c2);
      } else {
        leave_sums<kLanes>(c1, c2, red[walk.group][k & 1]);
        group_sync<kLanes>(walk.group);
        take_sums<kLanes>(c1, c2, red[walk.group][k & 1]);
      }
      if constexpr (kCluster > 1) {
        // (the bytes of the row after the next go to this row's barrier: they are sent by a block
        // that has met the next row's, which this block sends after all of it has met this row's)
        uint64_t* bar = &meet[walk.group].bar[k & 1];
        uint64_t* sums = meet[walk.group].sums[k & 1];
        if (t == 0 && stop < 0) {
          mbar_arrive_expect_tx(bar, 8 * kCluster);
#pragma unroll
          for (int r = 0; r < kCluster; ++r)
            store_async_u64(mapa_shared(smem_u32(sums + rank), r), pair(c1, c2),
                            mapa_shared(smem_u32(bar), r));
        }
        const uint32_t parity = static_cast<uint32_t>(k / 2) & 1u;
        if (!mbar_try_wait_cluster(smem_u32(bar), parity) && stop < 0 &&
            !mbar_wait<true>(bar, parity, st.wait_limit, &abort_flag, st.status, kSiteNormBwdMeet))
          stop = 2 * k + 1;
        uint64_t both = sums[0];
#pragma unroll
        for (int r = 1; r < kCluster; ++r) both = add2(both, sums[r]);
        unpair(both, c1, c2);
      }
      if (kBehind && t == 0 && stop < 0 && k + st.slots - 1 < walk.count)
        fill(k + st.slots - 1);
      c1 = quotient(c1, p.N, inv);
      c2 *= inv;
      const uint64_t r2 = pair(rstd, rstd), m1 = pair(-c1, -c1), m2 = pair(-c2, -c2);
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int n = (i * kLanes + t) * 8, q = kAgain ? 0 : i;
        if (!decltype(whole)::value && n >= cols) continue;
        if constexpr (kAgain) {
          float wv[8], none[8];
          kept_weights(ring, st.plane, n, wv);
          load_unit<kT>(at + st.at[0] + n * kSizeT, g[q]);
          load_unit<kS>(at + st.at[1] + n * kSizeS, h[q]);
          terms8<false>(mean, rstd, wv, g[q], h[q], p1, p2, none, none);
        }
        float d[8], f[8] = {};
        if (has_a) load_unit<kS>(at + st.at[2] + n * kSizeS, f);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const uint64_t x =
              fma2(pair(h[q][j], h[q][j + 1]), m2, add2(pair(g[q][j], g[q][j + 1]), m1));
          unpair(fma2(x, r2, pair(f[j], f[j + 1])), d[j], d[j + 1]);
        }
        if (has_s) store_unit<kS>(ds_row + n * kSizeS, d);
        if (has_x) {
          if constexpr (kDrop)
            drop8(p.drop,
                  kAgain ? drop_bits(p.drop, offset, row, col0 + n) : bits[kAgain ? 0 : i], d);
          store_unit<kT>(dx_row + n * kSizeT, d);
        }
      }
      if (last >= 0) {
        const float d = fmaf(rstd, fmaf(-h_last, c2, g_last - c1), f_last);
        if (has_s) store1<kS>(ds_row, last - col0, d);
        if (has_x)
          store1<kT>(dx_row, last - col0, kDrop ? drop1(p.drop, offset, row, last, d, 0.0f) : d);
      }
      if constexpr (!kBehind) {
        __syncwarp();
        if (t == 0 && stop < 0 && k + st.slots < walk.count) fill(k + st.slots);
      }
      mean = mean_next, rstd = rstd_next;
      ds_row += ds_step;
      dx_row += dx_step;
      if (++slot == st.slots) slot = 0, phase ^= 1u;
    }
  };
  if (__all_sync(0xffffffffu, ((kUnits - 1) * kLanes + t) * 8 < cols))
    walk_rows(std::true_type{});
  else
    walk_rows(std::false_type{});
  if (t == 0 && stop >= 0 &&
      !drain_slots(st, walk.bars, stop / 2, min(walk.count, stop / 2 + st.slots - kBehind)))
    lost = 1;
  if constexpr (kCluster > 1) {
    Meeting<kCluster>& m = meet[walk.group];
    if (t == 0 && stop >= 0) {
#pragma unroll
      for (int r = 0; r < kCluster; ++r)
        st_shared_cluster_u32(mapa_shared(smem_u32(m.sent + rank), r),
                              static_cast<uint32_t>(stop + 1) / 2);
    }
    cluster_sync();
    // (a leader that met all its rows has had all that is sent to it)
    if (t == 0 && stop >= 0) drain_meeting(m, rank, st.status);
  }
  if (p.partial == nullptr) return;
  // one row of sums per block or cluster: the groups' go over their rings, and are added in order
  float* tot = reinterpret_cast<float*>(ring);
  const int width = (rank == kCluster - 1 ? p.N : col0 + cols) - col0;
  __syncthreads();
  const bool ring_free = lost == 0;  // (else a copy may land in it yet, and the sums are no use)
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    if (!ring_free) break;
    const float(&acc)[kUnits][8] = v ? sb : sw;
    float* to = tot + (walk.group * 2 + v) * width;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int n = (i * kLanes + t) * 8;
      if (n >= cols) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) to[n + j] = acc[i][j];
    }
    if (last >= 0) to[last - col0] = v ? sb_last : sw_last;
  }
  __syncthreads();
  const int rows = static_cast<int>(gridDim.x) / kCluster;
  float* out = p.partial + static_cast<long long>(blockIdx.x / kCluster) * p.N + col0;
  for (int n = threadIdx.x; n < width; n += kGroups * kLanes) {
    float dw = 0.0f, db = 0.0f;
#pragma unroll
    for (int r = 0; r < kGroups; ++r) {
      dw += tot[2 * r * width + n];
      db += tot[(2 * r + 1) * width + n];
    }
    if (p.join) {
      if (ring_free) tot[n] = dw, tot[width + n] = db;
    } else {
      out[n] = dw;
      out[static_cast<long long>(rows) * p.N + n] = db;
    }
  }
  if (kCluster == 1 && p.join) join_sums<kT>(p, tot, tot + width);
}

// Rows of any length and alignment, without the column sums: the row is read twice.
template <int kT, int kS, int kThreads, bool kDrop>
__global__ void __launch_bounds__(kThreads) layer_norm_bwd_any_kernel(const NormBwdParams p) {
  __shared__ __align__(16) float2 red[kThreads / 32];
  grid_dependency_wait();
  grid_dependents_launch();
  const long long row = blockIdx.x;
  const bool vec = p.vec != 0;
  const uint64_t offset = kDrop ? drop_offset(p.drop) : 0;
  const float mean = p.mean[row], rstd = p.rstd[row];
  uint64_t p1 = 0, p2 = 0;
  float g[8] = {}, h[8] = {}, none[8];
  auto load = [&](auto type, const char* at, int n) {
    constexpr int kType = decltype(type)::value;
    return vec ? load8<kType>(at, n, p.N, true) : load8_shifted<kType>(at, n, p.N);
  };
  using T = std::integral_constant<int, kT>;
  using S = std::integral_constant<int, kS>;
  auto terms = [&](int n) {
    float w[8];
    load_vec8<kT>(p.w, n, p.N, p.w_f32, 1.0f, w);
    unpack8<kT>(load(T{}, row_at<kT>(p.dY, row, p.lddy), n), g);
    unpack8<kS>(load(S{}, row_at<kS>(p.S, row, p.lds), n), h);
    fill_past(h, n, p.N, mean);
    terms8<false>(mean, rstd, w, g, h, p1, p2, none, none);
  };
  for (long long n = threadIdx.x * 8; n < p.N; n += kThreads * 8) terms(static_cast<int>(n));
  float c1 = sum2(p1), c2 = sum2(p2);
  const float inv = 1.0f / static_cast<float>(p.N);
  leave_sums<kThreads>(c1, c2, red);
  __syncthreads();
  take_sums<kThreads>(c1, c2, red);
  c1 = quotient(c1, p.N, inv);
  c2 *= inv;
  char* ds_row = row_at<kS>(p.dS, row, p.ldds);
  char* dx_row = row_at<kT>(p.dX, row, p.lddx);
  // (the lanes of a warp stay together for the stores)
  for (long long m = threadIdx.x / 32 * 256; m < p.N; m += kThreads * 8) {
    const int n = static_cast<int>(m) + static_cast<int>(threadIdx.x) % 32 * 8;
    const bool there = n < p.N;
    Raw8<kS> a = {};
    if (there) {
      terms(n);
      if (p.A != nullptr) a = load(S{}, row_at<kS>(p.A, row, p.lda), n);
    }
    float d[8];
    slopes8<kS>(p, rstd, c1, c2, a, g, h, d);
    if (p.dS != nullptr) store8_warp<kS>(ds_row, n, p.N, vec, there, d);
    if (p.dX != nullptr) {
      if constexpr (kDrop) drop8(p.drop, drop_bits(p.drop, offset, row, n), d);
      store8_warp<kT>(dx_row, n, p.N, vec, there, d);
    }
  }
}

// Column sums over chunks of rows: a thread keeps eight columns and walks down every eighth
// row of the block's chunk.
template <int kT, int kS>
__global__ void __launch_bounds__(256) layer_norm_columns_kernel(const NormBwdParams p,
                                                                 int rows_per_chunk) {
  __shared__ float tot[8][256];
  grid_dependency_wait();
  grid_dependents_launch();
  const int lane = threadIdx.x % 32, sub = threadIdx.x / 32;
  const long long n0 = static_cast<long long>(blockIdx.x) * 256 + lane * 8;
  const long long r0 = static_cast<long long>(blockIdx.y) * rows_per_chunk;
  const long long r1 = min(static_cast<long long>(p.M), r0 + rows_per_chunk);
  const bool vec = p.vec != 0;
  float sw[8] = {}, sb[8] = {};
  if (n0 < p.N) {
    const int n = static_cast<int>(n0);
#pragma unroll 4
    for (long long row = r0 + sub; row < r1; row += 8) {
      const char* y_row = row_at<kT>(p.dY, row, p.lddy);
      const char* s_row = row_at<kS>(p.S, row, p.lds);
      const Raw8<kT> y = vec ? load8<kT>(y_row, n, p.N, true) : load8_shifted<kT>(y_row, n, p.N);
      const Raw8<kS> s = vec ? load8<kS>(s_row, n, p.N, true) : load8_shifted<kS>(s_row, n, p.N);
      const float mean = p.mean[row], rstd = p.rstd[row];
      float g[8], h[8];
      unpack8<kT>(y, g);
      unpack8<kS>(s, h);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sw[j] += g[j] * ((h[j] - mean) * rstd);
        sb[j] += g[j];
      }
    }
  }
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) tot[sub][lane * 8 + j] = v ? sb[j] : sw[j];
    __syncthreads();
    const long long n = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    float sum = 0.0f;
#pragma unroll
    for (int r = 0; r < 8; ++r) sum += tot[r][threadIdx.x];
    if (n < p.N)
      p.partial[(static_cast<long long>(v) * gridDim.y + blockIdx.y) * p.N + n] = sum;
  }
}

// Narrow rows: kLanes threads to a row, a unit to a thread, several rows at a time so that their
// loads and sums overlap (as many as 128 registers hold).  Rows of any alignment.
constexpr int kNarrowThreads = 512;
template <int kS>
constexpr int kNarrowRowsOf = kS == IGC_F32 ? 2 : 4;

template <int kT, int kS, int kLanes, bool kDrop>
__global__ void __launch_bounds__(kNarrowThreads, 1)
    layer_norm_bwd_narrow_kernel(const NormBwdParams p) {
  constexpr int kGroups = kNarrowThreads / kLanes, kNarrowRows = kNarrowRowsOf<kS>;
  __shared__ float tot[2][kGroups][kLanes * 8];
  grid_dependency_wait();
  grid_dependents_launch();
  const int t = threadIdx.x % kLanes, group = threadIdx.x / kLanes, n = t * 8;
  const bool vec = p.vec != 0;
  const uint64_t offset = kDrop ? drop_offset(p.drop) : 0;
  const float inv = 1.0f / static_cast<float>(p.N);
  float w[8], sw[8] = {}, sb[8] = {};
  load_vec8<kT>(p.w, n, p.N, p.w_f32, 1.0f, w);
  const long long step = static_cast<long long>(gridDim.x) * kGroups;
  // whole: no lane of the warp has a unit that the row's end cuts (65536 x 200 bf16 with dropout:
  // 35.5 us, 37.3 where every unit looks)
  auto walk_rows = [&](auto whole) {
    // (all groups of a warp go as often as the one with most rows)
    for (long long base = static_cast<long long>(blockIdx.x) * kGroups +
                          group / (32 / kLanes) * (32 / kLanes);
         base < p.M; base += step * kNarrowRows) {
      Raw8<kT> y[kNarrowRows];
      Raw8<kS> s[kNarrowRows], a[kNarrowRows];
      float mean[kNarrowRows], rstd[kNarrowRows];
#pragma unroll
      for (int r = 0; r < kNarrowRows; ++r) {
        const long long row = base + r * step + group % (32 / kLanes);
        y[r] = {}, s[r] = {}, a[r] = {};
        mean[r] = rstd[r] = 0.0f;
        if (row >= p.M || n >= p.N) continue;
        y[r] = load8<kT>(row_at<kT>(p.dY, row, p.lddy), n, p.N, vec);
        s[r] = load8<kS>(row_at<kS>(p.S, row, p.lds), n, p.N, vec);
        if (p.A != nullptr) a[r] = load8<kS>(row_at<kS>(p.A, row, p.lda), n, p.N, vec);
        mean[r] = p.mean[row], rstd[r] = p.rstd[row];
      }
#pragma unroll
      for (int r = 0; r < kNarrowRows; ++r) {
        const long long row = base + r * step + group % (32 / kLanes);
        float g[8], h[8];
        uint64_t p1 = 0, p2 = 0;
        unpack8<kT>(y[r], g);
        unpack8<kS>(s[r], h);
        if constexpr (!decltype(whole)::value) fill_past(h, n, p.N, mean[r]);
        terms8<true>(mean[r], rstd[r], w, g, h, p1, p2, sw, sb);
        float c1 = sum2(p1), c2 = sum2(p2);
        lane_sums<kLanes>(c1, c2);
        if (row >= p.M || n >= p.N) continue;
        float d[8];
        slopes8<kS>(p, rstd[r], quotient(c1, p.N, inv), c2 * inv, a[r], g, h, d);
        if (p.dS != nullptr) store8<kS>(row_at<kS>(p.dS, row, p.ldds), n, p.N, vec, d);
        if (p.dX != nullptr) {
          if constexpr (kDrop) drop8(p.drop, drop_bits(p.drop, offset, row, n), d);
          store8<kT>(row_at<kT>(p.dX, row, p.lddx), n, p.N, vec, d);
        }
      }
    }
  };
  if (__all_sync(0xffffffffu, n + 8 <= p.N || n >= p.N))
    walk_rows(std::true_type{});
  else
    walk_rows(std::false_type{});
  if (p.partial == nullptr) return;
  // one row of sums per block: the groups' are added in order
#pragma unroll
  for (int j = 0; j < 8; ++j) tot[0][group][n + j] = sw[j], tot[1][group][n + j] = sb[j];
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * kLanes * 8; c += kNarrowThreads) {
    const int v = c / (kLanes * 8), col = c % (kLanes * 8);
    if (col >= p.N) continue;
    float sum = 0.0f;
#pragma unroll 16
    for (int r = 0; r < kGroups; ++r) sum += tot[v][r][col];
    if (p.join)
      tot[v][0][col] = sum;
    else
      p.partial[(static_cast<long long>(v) * gridDim.x + blockIdx.x) * p.N + col] = sum;
  }
  if (p.join) join_sums<kT>(p, tot[0][0], tot[1][0]);
}

// Blocks of a launch whose blocks have `rows` rows side by side: as many as there is work for, at
// most `most`.  *join (if not null): whether they are one cluster that adds its blocks' sums, as
// where none then takes more than `once` rows, which take as long as one (64 x 1000 bf16: 12.9 us
// a call, 6.9 on the device, as two launches 15.2 and 6.5; with four times the rows 10 on the
// device).
inline int norm_bwd_blocks(const NormBwdParams& p, int64_t rows, int64_t once, int64_t most,
                           bool* join) {
  if (join != nullptr && p.partial != nullptr && p.M <= kJoinBlocks * once) {
    *join = true;
    most = kJoinBlocks;
  }
  const int64_t all = (static_cast<int64_t>(p.M) + rows - 1) / rows;
  if (most > kMaxPartials) most = kMaxPartials;
  return static_cast<int>(all < most ? all : most);
}

template <int kT, int kS, int kLanes>
int launch_narrow(const DeviceInfo& dev, NormBwdParams p, bool drop, int* blocks,
                  cudaStream_t stream) {
  constexpr int kRows = kNarrowThreads / kLanes;
  bool join = false;
  *blocks = norm_bwd_blocks(p, kRows, kRows * kNarrowRowsOf<kS>, dev.sm_count, &join);
  p.join = join;
  const int rc = launch_clusters(drop ? layer_norm_bwd_narrow_kernel<kT, kS, kLanes, true>
                                      : layer_norm_bwd_narrow_kernel<kT, kS, kLanes, false>,
                                 *blocks, join ? *blocks : 1, kNarrowThreads, 0, stream, p);
  if (join) *blocks = 0;
  return rc;
}

// *done: whether a block's shared memory holds two rows of every group.
template <int kT, int kS, int kLanes, int kUnits, int kCluster>
int stream_norm_bwd(const DeviceInfo& dev, NormBwdParams p, bool drop, int* blocks, bool* done,
                    cudaStream_t stream) {
  constexpr int kGroups = kNormBwdStreamMost / kLanes;
  auto kernel = drop ? layer_norm_bwd_stream_kernel<kT, kS, kLanes, kUnits, kCluster, true>
                     : layer_norm_bwd_stream_kernel<kT, kS, kLanes, kUnits, kCluster, false>;
  static StreamSetup setup[2];
  const int rc = stream_setup(setup[drop], kernel, dev, kCluster, kGroups * kLanes);
  if (rc != IGC_OK) return rc;
  RowStream st;
  const int64_t cols = (p.N / 8 + kCluster - 1) / kCluster * 8;
  const int sizes[kStreamMats] = {static_cast<int>(elem_size(kT)), static_cast<int>(elem_size(kS)),
                                  p.A != nullptr ? static_cast<int>(elem_size(kS)) : 0};
  *done = plan_stream(dev, cols, sizes, kGroups, &st);
  if (!*done) return IGC_OK;
  bool join = false;
  const int rows = norm_bwd_blocks(p, kGroups, kGroups, setup[drop].clusters[dev.device],
                                   kCluster == 1 ? &join : nullptr);
  p.join = join;
  *blocks = join ? 0 : rows;
  return launch_stream(kernel, rows * kCluster, join ? rows : kCluster, kGroups * kLanes, kGroups,
                       static_cast<size_t>(kGroups) * (cols + 8) * 8, stream, p, st);
}

// *blocks: rows of partial sums that it leaves (0: it has written dw and db).
template <int kT, int kS>
int run_norm_bwd(const DeviceInfo& dev, const NormBwdParams& p, bool drop, int* blocks,
                 cudaStream_t stream) {
  const long long units = (static_cast<long long>(p.N) + 7) / 8;
  if (units <= 8) return launch_narrow<kT, kS, 8>(dev, p, drop, blocks, stream);
  if (units <= 16) return launch_narrow<kT, kS, 16>(dev, p, drop, blocks, stream);
  if (units <= 32) return launch_narrow<kT, kS, 32>(dev, p, drop, blocks, stream);
  bool done = false;
  int rc = IGC_OK;
  if (!p.vec)
    done = false;
  else if (units <= 64)
    rc = stream_norm_bwd<kT, kS, 32, 2, 1>(dev, p, drop, blocks, &done, stream);
  else if (units <= 128)
    rc = stream_norm_bwd<kT, kS, 64, 2, 1>(dev, p, drop, blocks, &done, stream);
  else if (units <= 192)  // (32768 x 1536 bf16: five rows at once, 88 us; four of 128 threads 108)
    rc = stream_norm_bwd<kT, kS, 96, 2, 1>(dev, p, drop, blocks, &done, stream);
  else if (units <= 256)
    rc = stream_norm_bwd<kT, kS, 128, 2, 1>(dev, p, drop, blocks, &done, stream);
  else if (units <= 320)  // (16384 x 2500: three at once, 93 us; two of 256 threads 125)
    rc = stream_norm_bwd<kT, kS, 160, 2, 1>(dev, p, drop, blocks, &done, stream);
  else if (units <= 512)
    rc = stream_norm_bwd<kT, kS, 256, 2, 1>(dev, p, drop, blocks, &done, stream);
  // Three units to a thread where two rows at once then fit a block's or cluster's shared memory
  // and a wider form would leave a quarter of its threads without work (8192 x 6000: 94 us, one row
  // of 512 threads 108; 4096 x 12000: 102, clusters of four 125).
  else if (units <= 768)
    rc = stream_norm_bwd<kT, kS, 256, 3, 1>(dev, p, drop, blocks, &done, stream);
  else if (units > 1024 && units <= 1536)
    rc = stream_norm_bwd<kT, kS, 256, 3, 2>(dev, p, drop, blocks, &done, stream);
  else if (units > 2048 && units <= 12 * 256)
    rc = stream_norm_bwd<kT, kS, 256, 3, 4>(dev, p, drop, blocks, &done, stream);
  if (p.vec && !done && rc == IGC_OK && units > 512) {
    if (units <= 1024)
      rc = stream_norm_bwd<kT, kS, 512, 2, 1>(dev, p, drop, blocks, &done, stream);
    else if (units <= 2048)
      rc = stream_norm_bwd<kT, kS, 256, 2, 4>(dev, p, drop, blocks, &done, stream);
    else if (units <= 4096)
      rc = stream_norm_bwd<kT, kS, 256, 2, 8>(dev, p, drop, blocks, &done, stream);
  }
  if (done || rc != IGC_OK) return rc;
  if (p.dS != nullptr || p.dX != nullptr) {
    const dim3 grid(static_cast<unsigned>(p.M));
    rc = units <= 1024 ? launch_pdl(drop ? layer_norm_bwd_any_kernel<kT, kS, 128, true>
                                         : layer_norm_bwd_any_kernel<kT, kS, 128, false>,
                                    grid, dim3(128), 0, stream, p)
                       : launch_pdl(drop ? layer_norm_bwd_any_kernel<kT, kS, 512, true>
                                         : layer_norm_bwd_any_kernel<kT, kS, 512, false>,
                                    grid, dim3(512), 0, stream, p);
    if (rc != IGC_OK) return rc;
  }
  if (p.partial == nullptr) return IGC_OK;
  const int64_t col_blocks = (static_cast<int64_t>(p.N) + 255) / 256;
  int64_t chunks = (dev.sm_count * 8 + col_blocks - 1) / col_blocks;
  if (chunks > kMaxPartials) chunks = kMaxPartials;
  const int64_t rows = ((p.M + chunks - 1) / chunks + 7) / 8 * 8;
  chunks = (p.M + rows - 1) / rows;
  *blocks = static_cast<int>(chunks);
  return launch_pdl(layer_norm_columns_kernel<kT, kS>,
                    dim3(static_cast<unsigned>(col_blocks), static_cast<unsigned>(chunks)),
                    dim3(256), 0, stream, p, static_cast<int>(rows));
}

// By type of dY and of the residual stream (a file each: they compile side by side).
int layer_norm_bwd_f32(const DeviceInfo& dev, const NormBwdParams& p, bool drop, int* blocks,
                       cudaStream_t stream);
int layer_norm_bwd_f16(const DeviceInfo& dev, const NormBwdParams& p, bool drop, int* blocks,
                       cudaStream_t stream);
int layer_norm_bwd_f16_f32(const DeviceInfo& dev, const NormBwdParams& p, bool drop, int* blocks,
                           cudaStream_t stream);
int layer_norm_bwd_bf16(const DeviceInfo& dev, const NormBwdParams& p, bool drop, int* blocks,
                        cudaStream_t stream);
int layer_norm_bwd_bf16_f32(const DeviceInfo& dev, const NormBwdParams& p, bool drop, int* blocks,
                            cudaStream_t stream);

}  // namespace igc
