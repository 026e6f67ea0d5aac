// dX = sum_s D_s W_s: one contraction over the pre-activation gradients of linear_act
// (one segment) or gated_ffn (two).
#include "ffn_launch.cuh"

namespace igc {

namespace {

FfnProblem problem(const GradArgs& a) {
  FfnProblem q;
  q.M = a.M, q.N = a.K, q.K = a.N, q.dtype = a.dtype;
  q.segs = q.count_a = q.count_b = a.count;
  for (int i = 0; i < a.count; ++i) q.A[i] = a.D[i], q.B[i] = a.W[i];
  q.out[0] = a.dX;
  return q;
}

}  // namespace

int ffn_estimate_x(const DeviceInfo& dev, const GradArgs& a, GradEstimate* e) {
  return ffn_estimate<FfnOp::GradX>(dev, problem(a), e);
}

int ffn_grad_x(const DeviceInfo& dev, const GradArgs& a, bool late_wait, cudaStream_t stream) {
  FfnProblem q = problem(a);
  q.late_wait = late_wait, q.tiles_only = a.tiles_only;
  return ffn_launch<FfnOp::GradX>(dev, q, stream);
}

}  // namespace igc
