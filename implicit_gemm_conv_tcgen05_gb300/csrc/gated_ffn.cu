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
  if (!fits32(M) || !fits32(F) || !fits32(K)) return IGC_ERR_UNSUPPORTED;
  if (K > 0 && (!operand_ok(X, ldx) || !operand_ok(Wg, ldw) || !operand_ok(Wu, ldw)))
    return IGC_ERR_MISALIGNED;

  DeviceInfo dev;
  int rc = current_device(&dev);
  if (rc != IGC_OK) return rc;

  const Mat outs[3] = {{H, ldh, dtype}, {G, ldgu, dtype}, {U, ldgu, dtype}};
  if (K == 0) {
    PointwiseArgs a;
    a.M = M, a.N = F, a.dtype = dtype, a.act = act;
    a.bias[0] = bg, a.bias[1] = bu, a.bias_dtype = bias_dtype;
    for (int i = 0; i < 3; ++i) a.out[i] = outs[i];
    return ffn_bias_only(a, true, stream);
  }
  const Mat x{X, ldx, dtype}, w[2] = {{Wg, ldw, dtype}, {Wu, ldw, dtype}};
  if (M <= kSkinnyMaxM) {
    SkinnyParams p = {};
    p.M = static_cast<int>(M), p.N = static_cast<int>(F);
    p.act = act;
    p.bias0 = bg, p.bias1 = bu, p.bias_f32 = bias_dtype == IGC_F32;
    return ffn_launch_skinny<true>(dev, dtype, K, x, w, p, outs, 3, stream);
  }
  FfnParams p = {};
  p.M = static_cast<int>(M), p.N = static_cast<int>(F);
  p.kb_seg = static_cast<int>((K + kFfnKS - 1) / kFfnKS);
  p.segs = 1, p.srcs = 1;
  p.act = act;
  p.bias0 = bg, p.bias1 = bu, p.bias_f32 = bias_dtype == IGC_F32;
  return ffn_launch<FfnOp::Gated>(dev, dtype, 1, &x, M, K, 2, w, F, K, outs, 3, p, stream);
}
