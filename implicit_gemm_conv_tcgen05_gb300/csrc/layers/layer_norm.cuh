// Forward layer norm over the rows of S = R + drop(X): the kernels and their launch for one
// type of X and Y (kT) and one of R and S (kS).
//
// Bound by memory: X and R are read once, S and Y written once.  A row's S stays in the
// registers of its threads (units of eight columns), so that mean and variance are two sums
// over registers; the variance is that of the differences from the mean, which a large mean
// does not cancel.  Rows that no block's registers hold are read three times.
#pragma once

#include "layers_host.h"

namespace igc {

struct NormParams {
  int M, N, vec, w_f32;
  const void* X;
  const void* R;
  void* S;
  void* Y;
  long long ldx, ldr, lds, ldy;
  const void* w;
  const void* b;
  float* mean;
  float* rstd;
  float eps;
  Drop drop;
};

// S of eight columns; X and R are each loaded if they are there.
template <int kT, int kS, bool kDrop>
__device__ __forceinline__ void joined8(const NormParams& p, uint64_t offset, long long row, int n,
                                        bool vec, float (&s)[8]) {
  Raw8<kT> x;
  Raw8<kS> r;
  if (p.X != nullptr) x = load8<kT>(row_at<kT>(p.X, row, p.ldx), n, p.N, vec);
  if (p.R != nullptr) r = load8<kS>(row_at<kS>(p.R, row, p.ldr), n, p.N, vec);
  if (p.X != nullptr) {
    unpack8<kT>(x, s);
    if constexpr (kDrop) drop8(p.drop, offset, row, n, s);
    if (p.R != nullptr) {
      float f[8];
      unpack8<kS>(r, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += f[j];
    }
  } else {
    unpack8<kS>(r, s);
  }
}

// kLanes threads to a row, kUnits units of eight columns to a thread; rows of 32 threads share
// a block of four warps.
template <int kT, int kS, int kLanes, int kUnits, bool kDrop>
__global__ void __launch_bounds__(kLanes < 128 ? 128 : kLanes)
    layer_norm_kernel(const NormParams p) {
  constexpr int kRows = kLanes < 128 ? 128 / kLanes : 1;
  __shared__ float red[2][kLanes / 32];
  grid_dependency_wait();
  grid_dependents_launch();
  const long long row = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / kLanes;
  if (kRows > 1 && row >= p.M) return;
  const int t = threadIdx.x % kLanes;
  const bool vec = p.vec != 0;
  const uint64_t offset = kDrop ? drop_offset(p.drop) : 0;
  float s[kUnits][8];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int n = (i * kLanes + t) * 8;
    if (n < p.N) {
      joined8<kT, kS, kDrop>(p, offset, row, n, vec, s[i]);
      sum += ((s[i][0] + s[i][1]) + (s[i][2] + s[i][3])) +
             ((s[i][4] + s[i][5]) + (s[i][6] + s[i][7]));
    }
  }
  const float mean = row_sum<kLanes>(sum, red[0]) / static_cast<float>(p.N);
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int n = (i * kLanes + t) * 8;
    if (n >= p.N) continue;
    if (p.S != nullptr) store8<kS>(row_at<kS>(p.S, row, p.lds), n, p.N, vec, s[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s[i][j] -= mean;
      if (n + j < p.N) sum += s[i][j] * s[i][j];
    }
  }
  const float var = row_sum<kLanes>(sum, red[1]) / static_cast<float>(p.N);
  const float rstd = 1.0f / sqrtf(var + p.eps);
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int n = (i * kLanes + t) * 8;
    if (n >= p.N) continue;
    float w[8], b[8];
    load_vec8<kT>(p.w, n, p.N, p.w_f32, 1.0f, w);
    load_vec8<kT>(p.b, n, p.N, p.w_f32, 0.0f, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[i][j] = s[i][j] * rstd * w[j] + b[j];
    store8<kT>(row_at<kT>(p.Y, row, p.ldy), n, p.N, vec, s[i]);
  }
  if (t == 0) {
    if (p.mean != nullptr) p.mean[row] = mean;
    if (p.rstd != nullptr) p.rstd[row] = rstd;
  }
}

// Rows of any length: S is formed again for each of the three passes.  (S may be R: it is
// stored in the last.)
template <int kT, int kS, bool kDrop>
__global__ void __launch_bounds__(1024) layer_norm_long_kernel(const NormParams p) {
  __shared__ float red[2][32];
  grid_dependency_wait();
  grid_dependents_launch();
  const long long row = blockIdx.x;
  const bool vec = p.vec != 0;
  const uint64_t offset = kDrop ? drop_offset(p.drop) : 0;
  float s[8], sum = 0.0f;
  for (long long n = threadIdx.x * 8; n < p.N; n += 8192) {
    joined8<kT, kS, kDrop>(p, offset, row, static_cast<int>(n), vec, s);
    sum += ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  }
  const float mean = row_sum<1024>(sum, red[0]) / static_cast<float>(p.N);
  sum = 0.0f;
  for (long long n = threadIdx.x * 8; n < p.N; n += 8192) {
    joined8<kT, kS, kDrop>(p, offset, row, static_cast<int>(n), vec, s);
    float q = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) q += n + j < p.N ? (s[j] - mean) * (s[j] - mean) : 0.0f;
    sum += q;
  }
  const float var = row_sum<1024>(sum, red[1]) / static_cast<float>(p.N);
  const float rstd = 1.0f / sqrtf(var + p.eps);
  for (long long m = threadIdx.x * 8; m < p.N; m += 8192) {
    const int n = static_cast<int>(m);
    joined8<kT, kS, kDrop>(p, offset, row, n, vec, s);
    if (p.S != nullptr) store8<kS>(row_at<kS>(p.S, row, p.lds), n, p.N, vec, s);
    float w[8], b[8];
    load_vec8<kT>(p.w, n, p.N, p.w_f32, 1.0f, w);
    load_vec8<kT>(p.b, n, p.N, p.w_f32, 0.0f, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = (s[j] - mean) * rstd * w[j] + b[j];
    store8<kT>(row_at<kT>(p.Y, row, p.ldy), n, p.N, vec, s);
  }
  if (threadIdx.x == 0) {
    if (p.mean != nullptr) p.mean[row] = mean;
    if (p.rstd != nullptr) p.rstd[row] = rstd;
  }
}

template <int kT, int kS, int kLanes, int kUnits>
int launch_norm(const NormParams& p, bool drop, cudaStream_t stream) {
  constexpr int kRows = kLanes < 128 ? 128 / kLanes : 1;
  const unsigned blocks = static_cast<unsigned>((static_cast<long long>(p.M) + kRows - 1) / kRows);
  return launch_pdl(drop ? layer_norm_kernel<kT, kS, kLanes, kUnits, true>
                         : layer_norm_kernel<kT, kS, kLanes, kUnits, false>,
                    dim3(blocks), dim3(kLanes * kRows), 0, stream, p);
}

template <int kT, int kS>
int run_norm(const NormParams& p, bool drop, cudaStream_t stream) {
  const long long units = (static_cast<long long>(p.N) + 7) / 8;
  if (units <= 32) return launch_norm<kT, kS, 32, 1>(p, drop, stream);
  if (units <= 64) return launch_norm<kT, kS, 32, 2>(p, drop, stream);
  if (units <= 128) return launch_norm<kT, kS, 32, 4>(p, drop, stream);
  if (units <= 256) return launch_norm<kT, kS, 128, 2>(p, drop, stream);
  if (units <= 512) return launch_norm<kT, kS, 256, 2>(p, drop, stream);
  if (units <= 1024) return launch_norm<kT, kS, 512, 2>(p, drop, stream);
  if (units <= 2048) return launch_norm<kT, kS, 512, 4>(p, drop, stream);
  return launch_pdl(drop ? layer_norm_long_kernel<kT, kS, true>
                         : layer_norm_long_kernel<kT, kS, false>,
                    dim3(static_cast<unsigned>(p.M)), dim3(1024), 0, stream, p);
}

// By type (layer_norm_f32.cu, layer_norm_f16.cu, layer_norm_bf16.cu).
int layer_norm_f32(const NormParams& p, bool drop, cudaStream_t stream);
int layer_norm_f16(const NormParams& p, int s_dtype, bool drop, cudaStream_t stream);
int layer_norm_bf16(const NormParams& p, int s_dtype, bool drop, cudaStream_t stream);

}  // namespace igc
