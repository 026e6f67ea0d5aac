// dW_s = D_s^T X: the weight gradients of linear_act (one matrix) or gated_ffn (two,
// in one launch).
#include "ffn_launch.cuh"

namespace igc {

namespace {

FfnProblem problem(const GradArgs& a) {
  FfnProblem q;
  q.M = a.N, q.N = a.K, q.K = a.M, q.dtype = a.dtype;
  q.srcs = q.count_a = a.count;
  for (int i = 0; i < a.count; ++i) q.A[i] = a.D[i], q.out[i] = a.dW[i];
  q.B[0] = a.X;
  return q;
}

}  // namespace

int ffn_estimate_w(const DeviceInfo& dev, const GradArgs& a, GradEstimate* e) {
  return ffn_estimate<FfnOp::GradW>(dev, problem(a), e);
}

int ffn_grad_w(const DeviceInfo& dev, const GradArgs& a, bool late_wait, cudaStream_t stream) {
  FfnProblem q = problem(a);
  q.late_wait = late_wait, q.tiles_only = a.tiles_only;
  return ffn_launch<FfnOp::GradW>(dev, q, stream);
}

}  // namespace igc
