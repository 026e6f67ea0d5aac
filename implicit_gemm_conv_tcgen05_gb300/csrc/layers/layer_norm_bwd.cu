// Entry point of layer_norm_backward (the kernels: layer_norm_bwd.cuh) and the sum of the
// blocks' column sums.
#include "layer_norm_bwd.cuh"

namespace igc {

namespace {

// out[v][n] = sum over blocks of partial[v][block][n]; blockIdx.y = v (0: dw, 1: db).
__global__ void __launch_bounds__(1024)
    norm_sums_kernel(const float* partial, int blocks, int N, void* dw, void* db, int f32,
                     int bf16) {
  __shared__ float red[32][33];
  grid_dependency_wait();
  grid_dependents_launch();
  void* out = blockIdx.y ? db : dw;
  if (out == nullptr) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long n = static_cast<long long>(blockIdx.x) * 32 + lane;
  const float* from = partial + static_cast<long long>(blockIdx.y) * blocks * N + n;
  float sum = 0.0f;
  if (n < N) {
#pragma unroll 8
    for (int b = warp; b < blocks; b += 32) sum += from[static_cast<long long>(b) * N];
  }
  red[warp][lane] = sum;
  __syncthreads();
  // (a warp adds the 32 sums of one column)
  sum = warp_sum_all(red[lane][warp]);
  const long long m = static_cast<long long>(blockIdx.x) * 32 + warp;
  if (lane == 0 && m < N) {
    if (f32)
      static_cast<float*>(out)[m] = sum;
    else
      store16(out, m, sum, bf16 != 0);
  }
}

}  // namespace

}  // namespace igc

using namespace igc;

extern "C" {

size_t layer_norm_backward_workspace_size(int64_t M, int64_t N) {
  if (M < 0 || N < 0) return 0;
  return static_cast<size_t>(2) * static_cast<size_t>(M < kMaxPartials ? M : kMaxPartials) *
         static_cast<size_t>(N) * sizeof(float);
}

int layer_norm_backward(int64_t M, int64_t N, int dtype, const void* dY, int64_t lddy,
                        const void* S, int64_t lds, int s_dtype, const float* mean,
                        const float* rstd, const void* w, int w_dtype, const void* A, int64_t lda,
                        double p, uint64_t seed, uint64_t offset, const uint64_t* step, void* dS,
                        int64_t ldds, void* dX, int64_t lddx, void* dw, void* db, int dw_dtype,
                        void* workspace, size_t workspace_bytes, igc_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (M < 0 || N < 1 || !is_type(dtype) || !is_type_or_f32(s_dtype, dtype) ||
      !is_type_or_f32(w_dtype, dtype) || !is_type_or_f32(dw_dtype, dtype))
    return IGC_ERR_INVALID_ARG;
  NormBwdParams a = {};
  bool active = false;
  if (!make_drop(p, seed, offset, step, &a.drop, &active)) return IGC_ERR_INVALID_ARG;
  if (dS == nullptr && dX == nullptr && dw == nullptr && db == nullptr) return IGC_OK;
  if (!fits32(M) || !fits32(N)) return IGC_ERR_UNSUPPORTED;
  if ((dS != nullptr && ldds < N) || (dX != nullptr && lddx < N)) return IGC_ERR_INVALID_ARG;
  if (M > 0 && (dY == nullptr || S == nullptr || mean == nullptr || rstd == nullptr ||
                lddy < N || lds < N || (A != nullptr && lda < N)))
    return IGC_ERR_INVALID_ARG;
  if (is_any(dS, dY, S, mean, rstd, w, step, dX, dw, db) ||
      is_any(dX, dY, S, mean, rstd, w, step, A, dw, db) ||
      is_any(dw, dY, S, mean, rstd, w, step, A, db) || is_any(db, dY, S, mean, rstd, w, step, A) ||
      (dS != nullptr && dS == A && lda != ldds))
    return IGC_ERR_INVALID_ARG;
  if (!elements_aligned(Mat{dY, lddy, dtype}, Mat{S, lds, s_dtype}, Mat{A, lda, s_dtype},
                        Mat{dS, ldds, s_dtype}, Mat{dX, lddx, dtype}, Mat{mean, 0, IGC_F32},
                        Mat{rstd, 0, IGC_F32}, Mat{w, 0, w_dtype}, Mat{dw, 0, dw_dtype},
                        Mat{db, 0, dw_dtype}) ||
      reinterpret_cast<uintptr_t>(step) % 8 != 0)
    return IGC_ERR_MISALIGNED;
  const bool sums = dw != nullptr || db != nullptr;
  DeviceInfo dev;
  int rc = current_device(&dev);
  if (rc != IGC_OK) return rc;
  if (sums && M > 0 &&
      (workspace == nullptr || workspace_bytes < layer_norm_backward_workspace_size(M, N) ||
       reinterpret_cast<uintptr_t>(workspace) % 256 != 0))
    return IGC_ERR_WORKSPACE;
  int blocks = 0;
  if (M > 0) {
    a.M = static_cast<int>(M), a.N = static_cast<int>(N);
    a.vec = rows_vec(M, dY, lddy, dtype) && rows_vec(M, S, lds, s_dtype) &&
            rows_vec(M, A, lda, s_dtype) && rows_vec(M, dS, ldds, s_dtype) &&
            rows_vec(M, dX, lddx, dtype);
    a.w_f32 = w_dtype == IGC_F32;
    a.dY = dY, a.S = S, a.A = A, a.dS = dS, a.dX = dX;
    a.lddy = lddy, a.lds = lds, a.lda = lda, a.ldds = ldds, a.lddx = lddx;
    a.mean = mean, a.rstd = rstd, a.w = w;
    a.partial = sums ? static_cast<float*>(workspace) : nullptr;
    a.dw = dw, a.db = db, a.dw_f32 = dw_dtype == IGC_F32;
    active = active && dX != nullptr;
    const bool wide = s_dtype == IGC_F32;
    if (dtype == IGC_F32)
      rc = layer_norm_bwd_f32(dev, a, active, &blocks, stream);
    else if (dtype == IGC_F16)
      rc = wide ? layer_norm_bwd_f16_f32(dev, a, active, &blocks, stream)
                : layer_norm_bwd_f16(dev, a, active, &blocks, stream);
    else
      rc = wide ? layer_norm_bwd_bf16_f32(dev, a, active, &blocks, stream)
                : layer_norm_bwd_bf16(dev, a, active, &blocks, stream);
    if (rc != IGC_OK) return rc;
  }
  if (!sums || (M > 0 && blocks == 0)) return IGC_OK;
  return launch_pdl(norm_sums_kernel, dim3(static_cast<unsigned>((N + 31) / 32), 2), dim3(1024),
                    0, stream, static_cast<const float*>(workspace), blocks,
                    static_cast<int>(N), dw, db, dw_dtype == IGC_F32 ? 1 : 0,
                    dtype == IGC_BF16 ? 1 : 0);
}

}  // extern "C"
