// dX = sum_s D_s W_s: one contraction over the pre-activation gradients of linear_act
// (one segment) or gated_ffn (two).
#include "ffn_launch.cuh"

namespace igc {

int ffn_grad_x(const DeviceInfo& dev, int64_t M, int64_t N, int64_t K, int dtype, int count,
               const Mat* D, const Mat* W, const Mat& dX, cudaStream_t stream) {
  FfnParams p = {};
  p.M = static_cast<int>(M), p.N = static_cast<int>(K);
  p.kb_seg = static_cast<int>((N + kFfnKS - 1) / kFfnKS);
  p.segs = count, p.srcs = 1;
  return ffn_launch<FfnOp::GradX>(dev, dtype, count, D, M, N, count, W, N, K, &dX, 1, p, stream);
}

}  // namespace igc
