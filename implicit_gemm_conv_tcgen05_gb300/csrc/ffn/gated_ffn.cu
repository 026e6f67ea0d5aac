// gated_ffn: both projections of a gated feed-forward block, the activation and the
// product in one kernel.
#include "ffn_launch.cuh"

using namespace igc;

extern "C" int gated_ffn(int64_t M, int64_t F, int64_t K, int dtype, const void* X, int64_t ldx,
                         const void* Wg, const void* Wu, int64_t ldw, const void* bg,
                         const void* bu, int bias_dtype, int act, void* G, void* U, int64_t ldgu,
                         void* H, int64_t ldh, igc_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (M < 0 || F < 0 || K < 0 || !is_operand_type(dtype)) return IGC_ERR_INVALID_ARG;
  if ((bg != nullptr || bu != nullptr) && bias_dtype != IGC_F32 && bias_dtype != dtype)
    return IGC_ERR_INVALID_ARG;
  if (act < IGC_ACT_NONE || act > IGC_ACT_SILU) return IGC_ERR_INVALID_ARG;
  if (M == 0 || F == 0) return IGC_OK;
  if (H == nullptr || ldh < F) return IGC_ERR_INVALID_ARG;
  if ((G == nullptr) != (U == nullptr) || (G != nullptr && ldgu < F)) return IGC_ERR_INVALID_ARG;
  if (K > 0 && (X == nullptr || Wg == nullptr || Wu == nullptr || ldx < K || ldw < K))
    return IGC_ERR_INVALID_ARG;
  if (is_any(H, X, Wg, Wu, bg, bu, G, U) || is_any(G, X, Wg, Wu, bg, bu, U) ||
      is_any(U, X, Wg, Wu, bg, bu))
    return IGC_ERR_INVALID_ARG;  // outputs are no inputs
  if (!fits32(M) || !fits32(F) || !fits32(K)) return IGC_ERR_UNSUPPORTED;
  if (K > 0 && (!operand_ok(X, ldx) || !operand_ok(Wg, ldw) || !operand_ok(Wu, ldw)))
    return IGC_ERR_MISALIGNED;
  const Mat outs[3] = {{H, ldh, dtype}, {G, ldgu, dtype}, {U, ldgu, dtype}};
  if (!elements_aligned(outs[0], outs[1], outs[2], Mat{bg, F, bias_dtype},
                        Mat{bu, F, bias_dtype}))
    return IGC_ERR_MISALIGNED;

  DeviceInfo dev;
  int rc = current_device(&dev);
  if (rc != IGC_OK) return rc;

  if (K == 0) {
    PointwiseArgs a;
    a.M = M, a.N = F, a.dtype = dtype, a.act = act;
    a.bias[0] = bg, a.bias[1] = bu, a.bias_dtype = bias_dtype;
    for (int i = 0; i < 3; ++i) a.out[i] = outs[i];
    return ffn_bias_only(a, true, stream);
  }
  FfnProblem q;
  q.M = M, q.N = F, q.K = K, q.dtype = dtype;
  q.A[0] = {X, ldx, dtype};
  q.B[0] = {Wg, ldw, dtype}, q.B[1] = {Wu, ldw, dtype}, q.count_b = 2;
  for (int i = 0; i < 3; ++i) q.out[i] = outs[i];
  q.act = act, q.bias[0] = bg, q.bias[1] = bu, q.bias_dtype = bias_dtype;
  ProductPlan plan;
  rc = ffn_plan<FfnOp::Gated>(dev, q, &plan);
  return rc == IGC_OK ? ffn_launch<FfnOp::Gated>(dev, q, plan, stream) : rc;
}
