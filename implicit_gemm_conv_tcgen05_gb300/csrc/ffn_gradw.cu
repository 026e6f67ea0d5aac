// dW_s = D_s^T X: the weight gradients of linear_act (one matrix) or gated_ffn (two,
// their m-tiles in one launch).
#include "ffn_launch.cuh"

namespace igc {

int ffn_grad_w(const DeviceInfo& dev, int64_t M, int64_t N, int64_t K, int dtype, int count,
               const Mat* D, const Mat& X, const Mat* dW, cudaStream_t stream) {
  FfnParams p = {};
  p.M = static_cast<int>(N), p.N = static_cast<int>(K);
  p.kb_seg = static_cast<int>((M + kFfnKS - 1) / kFfnKS);
  p.segs = 1, p.srcs = count;
  return ffn_launch<FfnOp::GradW>(dev, dtype, count, D, M, N, 1, &X, M, K, dW, count, p, stream);
}

}  // namespace igc
