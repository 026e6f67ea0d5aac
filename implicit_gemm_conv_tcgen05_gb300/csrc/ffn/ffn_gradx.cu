// dX = sum_s D_s W_s: one contraction over the pre-activation gradients of linear_act
// (one segment) or gated_ffn (two).
#include "ffn_launch.cuh"

namespace igc {

int ffn_plan_x(const DeviceInfo& dev, const GradArgs& a, ProductPlan* plan) {
  return ffn_plan<FfnOp::GradX>(dev, grad_x_problem(a.M, a.N, a.K, a.dtype, a.count), plan);
}

int ffn_grad_x(const DeviceInfo& dev, const GradArgs& a, const ProductPlan& plan, bool late_wait,
               cudaStream_t stream) {
  FfnProblem q = grad_x_problem(a.M, a.N, a.K, a.dtype, a.count);
  for (int i = 0; i < a.count; ++i) q.A[i] = a.D[i], q.B[i] = a.W[i];
  q.out[0] = a.dX;
  q.late_wait = late_wait;
  return ffn_launch<FfnOp::GradX>(dev, q, plan, stream);
}

}  // namespace igc
