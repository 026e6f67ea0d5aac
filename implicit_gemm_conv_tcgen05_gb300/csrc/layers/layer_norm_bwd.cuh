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
// blocks' in order (no atomics).
#pragma once

#include "layers_host.h"

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
  Drop drop;
};

// Blocks whose partial sums the workspace has room for.
inline int64_t norm_bwd_max_blocks(int64_t N) { return N <= 1024 ? 1216 : 608; }

// dS and dX of eight columns from g, h and the row's sums.
template <int kT, int kS, bool kDrop>
__device__ __forceinline__ void grads8(const NormBwdParams& p, uint64_t offset, long long row,
                                       int n, bool vec, float rstd, float c1, float c2,
                                       const Raw8<kS>& a, const float (&g)[8],
                                       const float (&h)[8]) {
  float d[8], f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) d[j] = rstd * (g[j] - c1 - h[j] * c2);
  if (p.A != nullptr) {
    unpack8<kS>(a, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j] += f[j];
  }
  if (p.dS != nullptr) store8<kS>(row_at<kS>(p.dS, row, p.ldds), n, p.N, vec, d);
  if (p.dX != nullptr) {
    if constexpr (kDrop) drop8(p.drop, offset, row, n, d);
    store8<kT>(row_at<kT>(p.dX, row, p.lddx), n, p.N, vec, d);
  }
}

// kLanes threads to a row, kUnits units of eight columns to a thread.  kSums: with the column
// sums.
template <int kT, int kS, int kLanes, int kUnits, bool kDrop, bool kSums>
__global__ void __launch_bounds__(kLanes < 128 ? 128 : kLanes)
    layer_norm_bwd_kernel(const NormBwdParams p) {
  constexpr int kRows = kLanes < 128 ? 128 / kLanes : 1;
  constexpr int kCols = kLanes * kUnits * 8;
  __shared__ float red[2][2][kLanes / 32];
  grid_dependency_wait();
  grid_dependents_launch();
  const int t = threadIdx.x % kLanes;
  const bool vec = p.vec != 0;
  const uint64_t offset = kDrop ? drop_offset(p.drop) : 0;
  const float inv = 1.0f / static_cast<float>(p.N);
  float sw[kSums ? kUnits : 1][8] = {}, sb[kSums ? kUnits : 1][8] = {};
  int phase = 0;
  for (long long row = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / kLanes;
       row < p.M; row += static_cast<long long>(gridDim.x) * kRows, phase ^= 1) {
    const float mean = p.mean[row], rstd = p.rstd[row];
    float g[kUnits][8], h[kUnits][8];
    Raw8<kS> a[kUnits];
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int n = (i * kLanes + t) * 8;
      if (n >= p.N) continue;
      const Raw8<kT> y = load8<kT>(row_at<kT>(p.dY, row, p.lddy), n, p.N, vec);
      const Raw8<kS> s = load8<kS>(row_at<kS>(p.S, row, p.lds), n, p.N, vec);
      if (p.A != nullptr) a[i] = load8<kS>(row_at<kS>(p.A, row, p.lda), n, p.N, vec);
      float w[8];
      load_vec8<kT>(p.w, n, p.N, p.w_f32, 1.0f, w);
      unpack8<kT>(y, g[i]);
      unpack8<kS>(s, h[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[i][j] = (h[i][j] - mean) * rstd;
        if constexpr (kSums) {
          sw[i][j] += g[i][j] * h[i][j];
          sb[i][j] += g[i][j];
        }
        g[i][j] *= w[j];
        // (past the row's end dY and so g are 0)
        c1 += g[i][j];
        c2 += g[i][j] * h[i][j];
      }
    }
    // (the next row uses the other pair of arrays: no barrier after the reads)
    c1 = warp_sum_all(c1);
    c2 = warp_sum_all(c2);
    if constexpr (kLanes > 32) {
      if (threadIdx.x % 32 == 0) {
        red[phase][0][threadIdx.x / 32] = c1;
        red[phase][1][threadIdx.x / 32] = c2;
      }
      __syncthreads();
      c1 = c2 = 0.0f;
#pragma unroll
      for (int i = 0; i < kLanes / 32; ++i) {
        c1 += red[phase][0][i];
        c2 += red[phase][1][i];
      }
    }
    c1 *= inv;
    c2 *= inv;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int n = (i * kLanes + t) * 8;
      if (n < p.N)
        grads8<kT, kS, kDrop>(p, offset, row, n, vec, rstd, c1, c2, a[i], g[i], h[i]);
    }
  }
  if constexpr (kSums) {
    // one row of sums per block: the block's rows of threads add theirs in order
    __shared__ float tot[kRows > 1 ? kCols : 1];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      float(&acc)[kUnits][8] = v ? sb : sw;
      for (int r = 0; kRows > 1 && r < kRows; ++r) {
        __syncthreads();
        if (static_cast<int>(threadIdx.x) / kLanes == r) {
#pragma unroll
          for (int i = 0; i < kUnits; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float& at = tot[(i * kLanes + t) * 8 + j];
              at = r == 0 ? acc[i][j] : at + acc[i][j];
            }
        }
      }
      float* out = p.partial + (static_cast<long long>(v) * gridDim.x + blockIdx.x) * p.N;
      if constexpr (kRows > 1) {
        __syncthreads();
        for (int n = threadIdx.x; n < p.N; n += blockDim.x) out[n] = tot[n];
      } else {
        const bool whole = (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
          const int n = (i * kLanes + t) * 8;
          if (n < p.N)
            store8<IGC_F32>(reinterpret_cast<char*>(out), n, p.N, whole, acc[i]);
        }
      }
    }
  }
}

// Rows of any length, without the column sums: the row is read twice.
template <int kT, int kS, bool kDrop>
__global__ void __launch_bounds__(512) layer_norm_bwd_long_kernel(const NormBwdParams p) {
  __shared__ float red[2][16];
  grid_dependency_wait();
  grid_dependents_launch();
  const long long row = blockIdx.x;
  const bool vec = p.vec != 0;
  const uint64_t offset = kDrop ? drop_offset(p.drop) : 0;
  const float mean = p.mean[row], rstd = p.rstd[row];
  auto terms = [&](int n, float(&g)[8], float(&h)[8]) {
    const Raw8<kT> y = load8<kT>(row_at<kT>(p.dY, row, p.lddy), n, p.N, vec);
    const Raw8<kS> s = load8<kS>(row_at<kS>(p.S, row, p.lds), n, p.N, vec);
    float w[8];
    load_vec8<kT>(p.w, n, p.N, p.w_f32, 1.0f, w);
    unpack8<kT>(y, g);
    unpack8<kS>(s, h);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[j] = (h[j] - mean) * rstd;
      g[j] *= w[j];
    }
  };
  float g[8], h[8], c1 = 0.0f, c2 = 0.0f;
  for (long long n = threadIdx.x * 8; n < p.N; n += 512 * 8) {
    terms(static_cast<int>(n), g, h);
    float q1 = 0.0f, q2 = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      q1 += g[j];
      q2 += g[j] * h[j];
    }
    c1 += q1;
    c2 += q2;
  }
  const float inv = 1.0f / static_cast<float>(p.N);
  c1 = row_sum<512>(c1, red[0]) * inv;
  c2 = row_sum<512>(c2, red[1]) * inv;
  for (long long m = threadIdx.x * 8; m < p.N; m += 512 * 8) {
    const int n = static_cast<int>(m);
    terms(n, g, h);
    Raw8<kS> a = {};
    if (p.A != nullptr) a = load8<kS>(row_at<kS>(p.A, row, p.lda), n, p.N, vec);
    grads8<kT, kS, kDrop>(p, offset, row, n, vec, rstd, c1, c2, a, g, h);
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
      const Raw8<kT> y = load8<kT>(row_at<kT>(p.dY, row, p.lddy), n, p.N, vec);
      const Raw8<kS> s = load8<kS>(row_at<kS>(p.S, row, p.lds), n, p.N, vec);
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

template <int kT, int kS, int kLanes, int kUnits>
int launch_norm_bwd(const DeviceInfo& dev, const NormBwdParams& p, bool drop, int* blocks,
                    cudaStream_t stream) {
  constexpr int kRows = kLanes < 128 ? 128 / kLanes : 1;
  constexpr int kBlock = kLanes * kRows;
  const bool sums = p.partial != nullptr;
  // about 1024 threads an SM
  int64_t most = static_cast<int64_t>(dev.sm_count) * (kBlock >= 1024 ? 1 : 1024 / kBlock);
  if (most > norm_bwd_max_blocks(p.N)) most = norm_bwd_max_blocks(p.N);
  const int64_t all = (static_cast<int64_t>(p.M) + kRows - 1) / kRows;
  *blocks = static_cast<int>(all < most ? all : most);
  void (*kern)(NormBwdParams) =
      drop ? (sums ? layer_norm_bwd_kernel<kT, kS, kLanes, kUnits, true, true>
                   : layer_norm_bwd_kernel<kT, kS, kLanes, kUnits, true, false>)
           : (sums ? layer_norm_bwd_kernel<kT, kS, kLanes, kUnits, false, true>
                   : layer_norm_bwd_kernel<kT, kS, kLanes, kUnits, false, false>);
  return launch_pdl(kern, dim3(static_cast<unsigned>(*blocks)), dim3(kBlock), 0, stream, p);
}

// *blocks: rows of partial sums that it leaves.
template <int kT, int kS>
int run_norm_bwd(const DeviceInfo& dev, const NormBwdParams& p, bool drop, int* blocks,
                 cudaStream_t stream) {
  const long long units = (static_cast<long long>(p.N) + 7) / 8;
  if (units <= 32) return launch_norm_bwd<kT, kS, 32, 1>(dev, p, drop, blocks, stream);
  if (units <= 64) return launch_norm_bwd<kT, kS, 32, 2>(dev, p, drop, blocks, stream);
  if (units <= 128) return launch_norm_bwd<kT, kS, 128, 1>(dev, p, drop, blocks, stream);
  if (units <= 256) return launch_norm_bwd<kT, kS, 128, 2>(dev, p, drop, blocks, stream);
  if (units <= 512) return launch_norm_bwd<kT, kS, 256, 2>(dev, p, drop, blocks, stream);
  if (units <= 1024) return launch_norm_bwd<kT, kS, 512, 2>(dev, p, drop, blocks, stream);
  if (p.dS != nullptr || p.dX != nullptr) {
    const int rc = launch_pdl(drop ? layer_norm_bwd_long_kernel<kT, kS, true>
                                   : layer_norm_bwd_long_kernel<kT, kS, false>,
                              dim3(static_cast<unsigned>(p.M)), dim3(512), 0, stream, p);
    if (rc != IGC_OK) return rc;
  }
  if (p.partial == nullptr) return IGC_OK;
  const int64_t col_blocks = (static_cast<int64_t>(p.N) + 255) / 256;
  int64_t chunks = (dev.sm_count * 8 + col_blocks - 1) / col_blocks;
  if (chunks > norm_bwd_max_blocks(p.N)) chunks = norm_bwd_max_blocks(p.N);
  const int64_t rows = ((p.M + chunks - 1) / chunks + 7) / 8 * 8;
  chunks = (p.M + rows - 1) / rows;
  *blocks = static_cast<int>(chunks);
  return launch_pdl(layer_norm_columns_kernel<kT, kS>,
                    dim3(static_cast<unsigned>(col_blocks), static_cast<unsigned>(chunks)),
                    dim3(256), 0, stream, p, static_cast<int>(rows));
}

// By type (layer_norm_bwd_f32.cu, layer_norm_bwd_f16.cu, layer_norm_bwd_bf16.cu).
int layer_norm_bwd_f32(const DeviceInfo& dev, const NormBwdParams& p, bool drop, int* blocks,
                       cudaStream_t stream);
int layer_norm_bwd_f16(const DeviceInfo& dev, const NormBwdParams& p, int s_dtype, bool drop,
                       int* blocks, cudaStream_t stream);
int layer_norm_bwd_bf16(const DeviceInfo& dev, const NormBwdParams& p, int s_dtype, bool drop,
                        int* blocks, cudaStream_t stream);

}  // namespace igc
