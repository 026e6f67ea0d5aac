// Forward layer norm over the rows of S = R + drop(X): the kernels and their launch for one
// type of X and Y (kT) and one of R and S (kS).
//
// Bound by memory: X and R are read once, S and Y written once.  A row's S stays in the
// registers of its threads (units of eight columns), so that mean and variance are two sums
// over registers; the variance is that of the differences from the mean, which a large mean
// does not cancel: only the roundings of its sum are left in them (16384 x 4096 bf16 with dropout
// and residual: 87 us, 537 MB at 6.2 TB/s).  Rows that no block's registers hold are read three
// times.
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

// S of eight columns from X and R, where each is there.
template <int kT, int kS, bool kDrop>
__device__ __forceinline__ void join8(const NormParams& p, uint64_t offset, long long row, int n,
                                      const Raw8<kT>& x, const Raw8<kS>& r, float (&s)[8]) {
  if (p.X == nullptr) {
    unpack8<kS>(r, s);
    return;
  }
  float f[8] = {};
  unpack8<kT>(x, s);
  if (p.R != nullptr) unpack8<kS>(r, f);
  if constexpr (kDrop) {
    drop8(p.drop, drop_bits(p.drop, offset, row, n), s, f);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      unpair(add2(pair(s[2 * j], s[2 * j + 1]), pair(f[2 * j], f[2 * j + 1])), s[2 * j],
             s[2 * j + 1]);
  }
}

// s less the mean; returns the sum of the squares.
__device__ __forceinline__ float center8(float (&s)[8], float mean, int n, int N) {
  fill_past(s, n, N, mean);  // (what lies past the row's end is to differ by nothing)
  const uint64_t m = pair(-mean, -mean);
  uint64_t q = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t d = add2(pair(s[2 * j], s[2 * j + 1]), m);
    q = fma2(d, d, q);
    unpair(d, s[2 * j], s[2 * j + 1]);
  }
  return sum2(q);
}

// Y of eight columns from the differences from the mean.
template <int kT>
__device__ __forceinline__ void affine8(const NormParams& p, float rstd, int n, float (&s)[8]) {
  float w[8], b[8];
  load_vec8<kT>(p.w, n, p.N, p.w_f32, 1.0f, w);
  load_vec8<kT>(p.b, n, p.N, p.w_f32, 0.0f, b);
  const uint64_t r = pair(rstd, rstd);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t d = mul2(pair(s[2 * j], s[2 * j + 1]), r);
    unpair(fma2(d, pair(w[2 * j], w[2 * j + 1]), pair(b[2 * j], b[2 * j + 1])), s[2 * j],
           s[2 * j + 1]);
  }
}

template <int kT, int kS, bool kDrop>
__device__ __forceinline__ void joined8(const NormParams& p, uint64_t offset, long long row, int n,
                                        bool vec, float (&s)[8]) {
  Raw8<kT> x;
  Raw8<kS> r;
  const char* x_row = row_at<kT>(p.X, row, p.ldx);
  const char* r_row = row_at<kS>(p.R, row, p.ldr);
  if (vec) {
    if (p.X != nullptr) x = load8<kT>(x_row, n, p.N, true);
    if (p.R != nullptr) r = load8<kS>(r_row, n, p.N, true);
  } else {
    if (p.X != nullptr) x = load8_shifted<kT>(x_row, n, p.N);
    if (p.R != nullptr) r = load8_shifted<kS>(r_row, n, p.N);
  }
  join8<kT, kS, kDrop>(p, offset, row, n, x, r, s);
}

// 1 / sqrt(x): the hardware's approximation and one step of Newton's on it.
__device__ __forceinline__ float rsqrt_step(float x) {
  const float y = rsqrtf(x);
  return y > 0.0f && y < INFINITY ? fmaf(0.5f * y, fmaf(-x * y, y, 1.0f), y) : y;
}

// Rows off 16-byte boundaries (load8_shifted, store8_warp), one to a block, four units to a thread.
template <int kT, int kS, int kLanes, bool kDrop>
__global__ void __launch_bounds__(kLanes) layer_norm_shifted_kernel(const NormParams p) {
  constexpr int kUnits = 4;
  __shared__ __align__(16) float red[2][kLanes / 32];
  grid_dependency_wait();
  grid_dependents_launch();
  const long long row = blockIdx.x;
  const uint64_t offset = kDrop ? drop_offset(p.drop) : 0;
  const float inv = 1.0f / static_cast<float>(p.N);
  const int n0 = static_cast<int>(threadIdx.x) * 8;
  float s[kUnits][8] = {};
  uint64_t total = 0;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    if (n0 + i * kLanes * 8 >= p.N) continue;
    joined8<kT, kS, kDrop>(p, offset, row, n0 + i * kLanes * 8, false, s[i]);
    total = add2(total, add2(add2(pair(s[i][0], s[i][1]), pair(s[i][2], s[i][3])),
                             add2(pair(s[i][4], s[i][5]), pair(s[i][6], s[i][7]))));
  }
  const float mean = quotient(row_sum<kLanes>(sum2(total), red[0]), p.N, inv);
  float squares = 0.0f;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int n = n0 + i * kLanes * 8;
    if (p.S != nullptr)
      store8_warp<kS>(row_at<kS>(p.S, row, p.lds), n, p.N, false, n < p.N, s[i]);
    if (n < p.N) squares += center8(s[i], mean, n, p.N);
  }
  const float var = row_sum<kLanes>(squares, red[1]) * inv;
  const float rstd = rsqrt_step(var + p.eps);
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int n = n0 + i * kLanes * 8;
    if (n < p.N) affine8<kT>(p, rstd, n, s[i]);
    store8_warp<kT>(row_at<kT>(p.Y, row, p.ldy), n, p.N, false, n < p.N, s[i]);
  }
  if (threadIdx.x == 0) {
    if (p.mean != nullptr) p.mean[row] = mean;
    if (p.rstd != nullptr) p.rstd[row] = rstd;
  }
}

// Rows of any length and alignment: S is formed again for each of the three passes.  (S may be
// R: it is stored in the last.)
template <int kT, int kS, bool kDrop>
__global__ void __launch_bounds__(1024) layer_norm_any_kernel(const NormParams p) {
  constexpr int kThreads = 1024;
  __shared__ __align__(16) float red[2][kThreads / 32];
  grid_dependency_wait();
  grid_dependents_launch();
  const long long row = blockIdx.x;
  const bool vec = p.vec != 0;
  const uint64_t offset = kDrop ? drop_offset(p.drop) : 0;
  float s[8], sum = 0.0f;
  for (long long n = threadIdx.x * 8; n < p.N; n += kThreads * 8) {
    joined8<kT, kS, kDrop>(p, offset, row, static_cast<int>(n), vec, s);
    sum += ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  }
  const float mean = row_sum<kThreads>(sum, red[0]) / static_cast<float>(p.N);
  sum = 0.0f;
  for (long long n = threadIdx.x * 8; n < p.N; n += kThreads * 8) {
    joined8<kT, kS, kDrop>(p, offset, row, static_cast<int>(n), vec, s);
    sum += center8(s, mean, static_cast<int>(n), p.N);
  }
  const float var = row_sum<kThreads>(sum, red[1]) / static_cast<float>(p.N);
  const float rstd = rsqrt_step(var + p.eps);
  // (the lanes of a warp stay together for the stores)
  for (long long m = threadIdx.x / 32 * 256; m < p.N; m += kThreads * 8) {
    const int n = static_cast<int>(m) + static_cast<int>(threadIdx.x) % 32 * 8;
    const bool there = n < p.N;
    if (there) joined8<kT, kS, kDrop>(p, offset, row, n, vec, s);
    if (p.S != nullptr) store8_warp<kS>(row_at<kS>(p.S, row, p.lds), n, p.N, vec, there, s);
    if (there) {
      (void)center8(s, mean, n, p.N);
      affine8<kT>(p, rstd, n, s);
    }
    store8_warp<kT>(row_at<kT>(p.Y, row, p.ldy), n, p.N, vec, there, s);
  }
  if (threadIdx.x == 0) {
    if (p.mean != nullptr) p.mean[row] = mean;
    if (p.rstd != nullptr) p.rstd[row] = rstd;
  }
}

// Rows that start on 16-byte boundaries, one to a group of kLanes threads, kUnits units to a
// thread, all loaded before the first is used.  A block to a row from 64 threads on: rows that
// share a block wait for one another (32768 x 1536 bf16 with dropout and residual: 65 us, two
// rows to a block 86).  Four units where rows are long, on 768 threads of 80 registers an SM
// (16384 x 4096: 87 us; on 640 threads of more registers 94; two units to twice the threads 96),
// three where that leaves fewer threads without, on 1024 (8192 x 6000: 72 us, on 768 80).
template <int kLanes, int kUnits>
struct NormRows {
  static constexpr int kBlock = kLanes < 64 ? 128 : kLanes, kGroups = kBlock / kLanes;
  static constexpr int kPerSm =
      kBlock > 256 ? 2 : (kUnits == 2 || kUnits == 3 ? 1024 : 768) / kBlock;
};

template <int kT, int kS, int kLanes, int kUnits, bool kDrop>
__global__ void __launch_bounds__(NormRows<kLanes, kUnits>::kBlock,
                                  NormRows<kLanes, kUnits>::kPerSm)
    layer_norm_rows_kernel(const NormParams p) {
  constexpr int kGroups = NormRows<kLanes, kUnits>::kGroups;
  constexpr int kSizeT = kT == IGC_F32 ? 4 : 2, kSizeS = kS == IGC_F32 ? 4 : 2;
  // few rows: w and b are loaded with the row, not after its sums (1 x 4096: 1.9 us, 2.1 after;
  // where rows fill the SMs their registers cost more: 65536 x 200 with dropout 31 instead of 27)
  constexpr bool kEarly = kUnits == 1 && kLanes >= 128;
  __shared__ __align__(16) float red[kGroups][2][(kLanes + 127) / 128 * 4];
  const int t = threadIdx.x % kLanes, group = threadIdx.x / kLanes, N8 = p.N / 8 * 8;
  const long long row = static_cast<long long>(blockIdx.x) * kGroups + group;
  grid_dependency_wait();
  grid_dependents_launch();
  // (rows of less than a warp: the warp stays together for its shuffles)
  if (kLanes >= 32 && kGroups > 1 && row >= p.M) return;
  const bool there = kLanes >= 32 || row < p.M;
  const bool has_x = p.X != nullptr, has_r = p.R != nullptr, has_s = p.S != nullptr;
  const uint64_t offset = kDrop ? drop_offset(p.drop) : 0;
  const float inv = 1.0f / static_cast<float>(p.N);
  const int last = there && N8 + t < p.N ? N8 + t : -1;
  const char* x_row = row_at<kT>(p.X, row, p.ldx);
  const char* r_row = row_at<kS>(p.R, row, p.ldr);
  char* s_row = row_at<kS>(p.S, row, p.lds);
  char* y_row = row_at<kT>(p.Y, row, p.ldy);
  auto one_row = [&](auto whole) {
    float s[kUnits][8], s_last = 0.0f;
    Raw8<kT> x[kUnits];
    Raw8<kS> r[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int n = (i * kLanes + t) * 8;
      if (!decltype(whole)::value && (n >= N8 || !there)) continue;
      if (has_x) x[i] = load8<kT>(x_row, n, n + 8, true);
      if (has_r) r[i] = load8<kS>(r_row, n, n + 8, true);
    }
    float w_early[8], b_early[8];
    if constexpr (kEarly) {
      load_vec8<kT>(p.w, t * 8, p.N, p.w_f32, 1.0f, w_early);
      load_vec8<kT>(p.b, t * 8, p.N, p.w_f32, 0.0f, b_early);
    }
    uint64_t sum = 0;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int n = (i * kLanes + t) * 8;
      if (!decltype(whole)::value && (n >= N8 || !there)) continue;
      float f[8] = {};
      if (has_r) unpack8<kS>(r[i], f);
      if constexpr (kDrop) {
        unpack8<kT>(x[i], s[i]);
        drop8(p.drop, drop_bits(p.drop, offset, row, n), s[i], f);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] = f[j];
        if (has_x) {
          unpack8<kT>(x[i], s[i]);
#pragma unroll
          for (int j = 0; j < 8; ++j) s[i][j] += f[j];
        }
      }
      sum = add2(sum, add2(add2(pair(s[i][0], s[i][1]), pair(s[i][2], s[i][3])),
                           add2(pair(s[i][4], s[i][5]), pair(s[i][6], s[i][7]))));
    }
    float total = sum2(sum);
    if (last >= 0) {
      const float x_last = has_x ? load1<kT>(x_row, last) : 0.0f;
      const float r_last = has_r ? load1<kS>(r_row, last) : 0.0f;
      s_last = kDrop ? drop1(p.drop, offset, row, last, x_last, r_last) : x_last + r_last;
      total += s_last;
    }
    const float mean = quotient(row_sum<kLanes>(total, red[group][0], group), p.N, inv);
    const uint64_t m = pair(-mean, -mean);
    uint64_t squares = 0;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int n = (i * kLanes + t) * 8;
      if (!decltype(whole)::value && (n >= N8 || !there)) continue;
      if (has_s) store_unit<kS>(s_row + n * kSizeS, s[i]);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const uint64_t d = add2(pair(s[i][j], s[i][j + 1]), m);
        squares = fma2(d, d, squares);
        unpair(d, s[i][j], s[i][j + 1]);
      }
    }
    total = sum2(squares);
    if (last >= 0) {
      if (has_s) store1<kS>(s_row, last, s_last);
      s_last -= mean;
      total = fmaf(s_last, s_last, total);
    }
    const float var = row_sum<kLanes>(total, red[group][1], group) * inv;
    const float rstd = rsqrt_step(var + p.eps);
    const uint64_t r2 = pair(rstd, rstd);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int n = (i * kLanes + t) * 8;
      if (!decltype(whole)::value && (n >= N8 || !there)) continue;
      float wv[8], bv[8];
      if constexpr (kEarly) {
#pragma unroll
        for (int j = 0; j < 8; ++j) wv[j] = w_early[j], bv[j] = b_early[j];
      } else {
        load_vec8<kT>(p.w, n, p.N, p.w_f32, 1.0f, wv);
        load_vec8<kT>(p.b, n, p.N, p.w_f32, 0.0f, bv);
      }
#pragma unroll
      for (int j = 0; j < 8; j += 2)
        unpair(fma2(mul2(pair(s[i][j], s[i][j + 1]), r2), pair(wv[j], wv[j + 1]),
                    pair(bv[j], bv[j + 1])),
               s[i][j], s[i][j + 1]);
      store_unit<kT>(y_row + n * kSizeT, s[i]);
    }
    if (last >= 0) {
      float wv = 1.0f, bv = 0.0f;
      if (p.w != nullptr) wv = load_vec(p.w, last, p.w_f32, kT == IGC_BF16);
      if (p.b != nullptr) bv = load_vec(p.b, last, p.w_f32, kT == IGC_BF16);
      store1<kT>(y_row, last, fmaf(s_last * rstd, wv, bv));
    }
    if (t == 0 && there) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
  };
  if (__all_sync(0xffffffffu, there && ((kUnits - 1) * kLanes + t) * 8 < N8))
    one_row(std::true_type{});
  else
    one_row(std::false_type{});
}

template <int kT, int kS, int kLanes, int kUnits>
int launch_rows(const NormParams& p, bool drop, cudaStream_t stream) {
  using Rows = NormRows<kLanes, kUnits>;
  const long long blocks = (static_cast<long long>(p.M) + Rows::kGroups - 1) / Rows::kGroups;
  return launch_pdl(drop ? layer_norm_rows_kernel<kT, kS, kLanes, kUnits, true>
                         : layer_norm_rows_kernel<kT, kS, kLanes, kUnits, false>,
                    dim3(static_cast<unsigned>(blocks)), dim3(Rows::kBlock), 0, stream, p);
}

// Three or four units to a thread, whichever leaves fewer of them without.
template <int kT, int kS, int kLanes>
int launch_long_rows(const NormParams& p, bool drop, cudaStream_t stream) {
  return p.N <= kLanes * 24 ? launch_rows<kT, kS, kLanes, 3>(p, drop, stream)
                            : launch_rows<kT, kS, kLanes, 4>(p, drop, stream);
}

template <int kT, int kS>
int run_norm(const DeviceInfo& dev, const NormParams& p, bool drop, cudaStream_t stream) {
  const long long units = (static_cast<long long>(p.N) + 7) / 8;
  // Few rows: a unit or two to a thread, so that a row is done sooner (on the device 1 x 1024 bf16
  // 1.4 us, 1 x 4096 1.9, 1 x 8192 2.8; with four units 2.6, 2.7 and 3.0).  As long as an SM holds
  // all its rows at once: 16 of 128 threads (600 x 1000: 2.0 us, 3.2 with four units; 2400 x 1000:
  // 4.6, 4.9), 8 of 256 (600 x 2048: 2.7, 3.2; 2400: 7.4, 8.1; 4800: 13.7, 11.7), two of 512 (333 x
  // 4096: 4.0, 3.5), and 4 where half of a row's threads have nothing (1200 x 512: 2.3, 2.3).
  const int at_once = units <= 64 ? 4 : units <= 128 ? 16 : units <= 256 ? 8 : 2;
  if (p.vec && units > 32 && p.M <= static_cast<long long>(at_once) * dev.sm_count) {
    if (units <= 128) return launch_rows<kT, kS, 128, 1>(p, drop, stream);
    if (units <= 256) return launch_rows<kT, kS, 256, 1>(p, drop, stream);
    if (units <= 512) return launch_rows<kT, kS, 512, 1>(p, drop, stream);
    if (units <= 1024) return launch_rows<kT, kS, 512, 2>(p, drop, stream);
  }
  if (p.vec) {
    if (units <= 8) return launch_rows<kT, kS, 8, 1>(p, drop, stream);
    if (units <= 16) return launch_rows<kT, kS, 16, 1>(p, drop, stream);
    if (units <= 32) return launch_rows<kT, kS, 32, 1>(p, drop, stream);
    if (units <= 64) return launch_rows<kT, kS, 32, 2>(p, drop, stream);
    if (units <= 128) return launch_long_rows<kT, kS, 32>(p, drop, stream);
    if (units <= 256) return launch_long_rows<kT, kS, 64>(p, drop, stream);
    if (units <= 512) return launch_long_rows<kT, kS, 128>(p, drop, stream);
    if (units <= 1024) return launch_long_rows<kT, kS, 256>(p, drop, stream);
    if (units <= 2048) return launch_long_rows<kT, kS, 512>(p, drop, stream);
  }
  const dim3 grid(static_cast<unsigned>(p.M));
  if (units <= 512)
    return launch_pdl(drop ? layer_norm_shifted_kernel<kT, kS, 128, true>
                           : layer_norm_shifted_kernel<kT, kS, 128, false>,
                      grid, dim3(128), 0, stream, p);
  if (units <= 1024)
    return launch_pdl(drop ? layer_norm_shifted_kernel<kT, kS, 256, true>
                           : layer_norm_shifted_kernel<kT, kS, 256, false>,
                      grid, dim3(256), 0, stream, p);
  if (units <= 2048)
    return launch_pdl(drop ? layer_norm_shifted_kernel<kT, kS, 512, true>
                           : layer_norm_shifted_kernel<kT, kS, 512, false>,
                      grid, dim3(512), 0, stream, p);
  return launch_pdl(drop ? layer_norm_any_kernel<kT, kS, true>
                         : layer_norm_any_kernel<kT, kS, false>,
                    grid, dim3(1024), 0, stream, p);
}

// By type of X and of the residual stream (a file each: they compile side by side).
int layer_norm_f32(const DeviceInfo& dev, const NormParams& p, bool drop, cudaStream_t stream);
int layer_norm_f16(const DeviceInfo& dev, const NormParams& p, bool drop, cudaStream_t stream);
int layer_norm_f16_f32(const DeviceInfo& dev, const NormParams& p, bool drop, cudaStream_t stream);
int layer_norm_bf16(const DeviceInfo& dev, const NormParams& p, bool drop, cudaStream_t stream);
int layer_norm_bf16_f32(const DeviceInfo& dev, const NormParams& p, bool drop,
                        cudaStream_t stream);

}  // namespace igc
