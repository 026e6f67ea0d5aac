// linear_act: a matrix product with bias, activation and residual in its epilogue.
#include "ffn_launch.cuh"

using namespace igc;

extern "C" int linear_act(int64_t M, int64_t N, int64_t K, int dtype, const void* X, int64_t ldx,
                          const void* W, int64_t ldw, const void* bias, int bias_dtype, int act,
                          const void* R, int64_t ldr, void* Z, int64_t ldz, void* Y, int64_t ldy,
                          int y_dtype, igc_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (M < 0 || N < 0 || K < 0 || !is_operand_type(dtype)) return IGC_ERR_INVALID_ARG;
  if (y_dtype != IGC_F32 && y_dtype != dtype) return IGC_ERR_INVALID_ARG;
  if (bias != nullptr && bias_dtype != IGC_F32 && bias_dtype != dtype) return IGC_ERR_INVALID_ARG;
  if (act < IGC_ACT_NONE || act > IGC_ACT_SILU) return IGC_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return IGC_OK;
  if (Y == nullptr || ldy < N || (R != nullptr && ldr < N) || (Z != nullptr && ldz < N))
    return IGC_ERR_INVALID_ARG;
  if (K > 0 && (X == nullptr || W == nullptr || ldx < K || ldw < K)) return IGC_ERR_INVALID_ARG;
  if (!fits32(M) || !fits32(N) || !fits32(K)) return IGC_ERR_UNSUPPORTED;
  if (K > 0 && (!operand_ok(X, ldx) || !operand_ok(W, ldw))) return IGC_ERR_MISALIGNED;

  DeviceInfo dev;
  int rc = current_device(&dev);
  if (rc != IGC_OK) return rc;

  const Mat outs[2] = {{Y, ldy, y_dtype}, {Z, ldz, dtype}};
  if (K == 0) {
    PointwiseArgs a;
    a.M = M, a.N = N, a.dtype = dtype, a.act = act;
    a.bias[0] = bias, a.bias_dtype = bias_dtype;
    a.R = {R, ldr, dtype};
    a.out[0] = outs[0], a.out[1] = outs[1];
    return ffn_bias_only(a, false, stream);
  }
  const Mat x{X, ldx, dtype}, w{W, ldw, dtype};
  if (M <= kSkinnyMaxM) {
    SkinnyParams p = {};
    p.M = static_cast<int>(M), p.N = static_cast<int>(N);
    p.act = act;
    p.bias0 = bias, p.bias_f32 = bias_dtype == IGC_F32;
    p.R = R, p.ldr = ldr, p.r_vec = rows_aligned(R, ldr, 2, 8);
    return ffn_launch_skinny<false>(dev, dtype, K, x, &w, p, outs, 2, stream);
  }
  FfnParams p = {};
  p.M = static_cast<int>(M), p.N = static_cast<int>(N);
  p.kb_seg = static_cast<int>((K + kFfnKS - 1) / kFfnKS);
  p.segs = 1, p.srcs = 1;
  p.act = act;
  p.bias0 = bias, p.bias_f32 = bias_dtype == IGC_F32;
  p.R = R, p.ldr = ldr, p.r_vec = rows_aligned(R, ldr, 2, 16);
  return ffn_launch<FfnOp::Linear>(dev, dtype, 1, &x, M, K, 1, &w, N, K, outs, 2, p, stream);
}
