// dW_s = D_s^T X: the weight gradients of linear_act (one matrix) or gated_ffn (two,
// in one launch).
#include "ffn_launch.cuh"

namespace igc {

int ffn_grad_w(const DeviceInfo& dev, int64_t M, int64_t N, int64_t K, int dtype, int count,
               const Mat* D, const Mat& X, const Mat* dW, bool late_wait,
               cudaStream_t stream) {
  FfnProblem q;
  q.late_wait = late_wait;
  q.M = N, q.N = K, q.K = M, q.dtype = dtype;
  q.srcs = q.count_a = count;
  for (int i = 0; i < count; ++i) q.A[i] = D[i], q.out[i] = dW[i];
  q.B[0] = X;
  return ffn_launch<FfnOp::GradW>(dev, q, stream);
}

}  // namespace igc
