// dW_s = D_s^T X: the weight gradients of linear_act (one matrix) or gated_ffn (two,
// in one launch).
#include "ffn_launch.cuh"

namespace igc {

int ffn_plan_w(const DeviceInfo& dev, const GradArgs& a, ProductPlan* plan) {
  return ffn_plan<FfnOp::GradW>(dev, grad_w_problem(a.M, a.N, a.K, a.dtype, a.count), plan);
}

int ffn_grad_w(const DeviceInfo& dev, const GradArgs& a, const ProductPlan& plan, bool late_wait,
               cudaStream_t stream) {
  FfnProblem q = grad_w_problem(a.M, a.N, a.K, a.dtype, a.count);
  for (int i = 0; i < a.count; ++i) q.A[i] = a.D[i], q.out[i] = a.dW[i];
  q.B[0] = a.X;
  q.late_wait = late_wait;
  return ffn_launch<FfnOp::GradW>(dev, q, plan, stream);
}

}  // namespace igc
