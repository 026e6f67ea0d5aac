// Entry point of layer_norm: checks and dispatch (the kernels: layer_norm.cuh).
#include "layer_norm.cuh"

using namespace igc;

extern "C" int layer_norm(int64_t M, int64_t N, int dtype, const void* X, int64_t ldx,
                          const void* R, int64_t ldr, int s_dtype, double p, uint64_t seed,
                          uint64_t offset, const uint64_t* step, const void* w, const void* b,
                          int w_dtype, float eps, void* S, int64_t lds, void* Y, int64_t ldy,
                          float* mean, float* rstd, igc_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (M < 0 || N < 1 || !is_type(dtype) || !is_type_or_f32(s_dtype, dtype) ||
      !is_type_or_f32(w_dtype, dtype) || !(eps >= 0.0f))
    return IGC_ERR_INVALID_ARG;
  NormParams a = {};
  bool active = false;
  if (!make_drop(p, seed, offset, step, &a.drop, &active)) return IGC_ERR_INVALID_ARG;
  if (M == 0) return IGC_OK;
  if (!fits32(M) || !fits32(N)) return IGC_ERR_UNSUPPORTED;
  if ((X == nullptr && R == nullptr) || Y == nullptr || ldy < N || (X != nullptr && ldx < N) ||
      (R != nullptr && ldr < N) || (S != nullptr && lds < N))
    return IGC_ERR_INVALID_ARG;
  if (is_any(Y, X, R, S, w, b, step, mean, rstd) || is_any(S, X, w, b, step, mean, rstd) ||
      is_any(mean, X, R, w, b, step, rstd) || is_any(rstd, X, R, w, b, step) ||
      (S != nullptr && S == R && lds != ldr))
    return IGC_ERR_INVALID_ARG;
  if (!elements_aligned(Mat{X, ldx, dtype}, Mat{R, ldr, s_dtype}, Mat{S, lds, s_dtype},
                        Mat{Y, ldy, dtype}, Mat{w, 0, w_dtype}, Mat{b, 0, w_dtype},
                        Mat{mean, 0, IGC_F32}, Mat{rstd, 0, IGC_F32}) ||
      reinterpret_cast<uintptr_t>(step) % 8 != 0)
    return IGC_ERR_MISALIGNED;
  DeviceInfo dev;
  const int rc = current_device(&dev);
  if (rc != IGC_OK) return rc;
  a.M = static_cast<int>(M), a.N = static_cast<int>(N);
  a.vec = rows_vec(M, X, ldx, dtype) && rows_vec(M, R, ldr, s_dtype) &&
          rows_vec(M, S, lds, s_dtype) && rows_vec(M, Y, ldy, dtype);
  a.w_f32 = w_dtype == IGC_F32;
  a.X = X, a.R = R, a.S = S, a.Y = Y;
  a.ldx = ldx, a.ldr = ldr, a.lds = lds, a.ldy = ldy;
  a.w = w, a.b = b, a.mean = mean, a.rstd = rstd, a.eps = eps;
  active = active && X != nullptr;
  const bool wide = s_dtype == IGC_F32;
  if (dtype == IGC_F32) return layer_norm_f32(dev, a, active, stream);
  if (dtype == IGC_F16)
    return wide ? layer_norm_f16_f32(dev, a, active, stream)
                : layer_norm_f16(dev, a, active, stream);
  return wide ? layer_norm_bf16_f32(dev, a, active, stream)
              : layer_norm_bf16(dev, a, active, stream);
}
