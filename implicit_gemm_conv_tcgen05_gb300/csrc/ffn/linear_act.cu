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
  // outputs are no inputs; the residual may be Y itself, element for element
  if (is_any(Y, X, W, bias, Z) || is_any(Z, X, W, bias, R)) return IGC_ERR_INVALID_ARG;
  if (R == Y && (ldr != ldy || y_dtype != dtype)) return IGC_ERR_INVALID_ARG;
  if (!fits32(M) || !fits32(N) || !fits32(K)) return IGC_ERR_UNSUPPORTED;
  if (K > 0 && (!operand_ok(X, ldx) || !operand_ok(W, ldw))) return IGC_ERR_MISALIGNED;
  const Mat outs[2] = {{Y, ldy, y_dtype}, {Z, ldz, dtype}};
  if (!elements_aligned(outs[0], outs[1], Mat{R, ldr, dtype}, Mat{bias, N, bias_dtype}))
    return IGC_ERR_MISALIGNED;

  DeviceInfo dev;
  int rc = current_device(&dev);
  if (rc != IGC_OK) return rc;

  if (K == 0) {
    PointwiseArgs a;
    a.M = M, a.N = N, a.dtype = dtype, a.act = act;
    a.bias[0] = bias, a.bias_dtype = bias_dtype;
    a.R = {R, ldr, dtype};
    a.out[0] = outs[0], a.out[1] = outs[1];
    return ffn_bias_only(a, false, stream);
  }
  FfnProblem q;
  q.M = M, q.N = N, q.K = K, q.dtype = dtype;
  q.A[0] = {X, ldx, dtype}, q.B[0] = {W, ldw, dtype};
  q.out[0] = outs[0], q.out[1] = outs[1];
  q.act = act, q.bias[0] = bias, q.bias_dtype = bias_dtype;
  q.R = {R, ldr, dtype};
  ProductPlan plan;
  rc = ffn_plan<FfnOp::Linear>(dev, q, &plan);
  return rc == IGC_OK ? ffn_launch<FfnOp::Linear>(dev, q, plan, stream) : rc;
}
