// dX = sum_s D_s W_s: one contraction over the pre-activation gradients of linear_act
// (one segment) or gated_ffn (two).
#include "ffn_launch.cuh"

namespace igc {

int ffn_grad_x(const DeviceInfo& dev, int64_t M, int64_t N, int64_t K, int dtype, int count,
               const Mat* D, const Mat* W, const Mat& dX, bool late_wait,
               cudaStream_t stream) {
  FfnProblem q;
  q.late_wait = late_wait;
  q.M = M, q.N = K, q.K = N, q.dtype = dtype;
  q.segs = q.count_a = q.count_b = count;
  for (int i = 0; i < count; ++i) q.A[i] = D[i], q.B[i] = W[i];
  q.out[0] = dX;
  return ffn_launch<FfnOp::GradX>(dev, q, stream);
}

}  // namespace igc
