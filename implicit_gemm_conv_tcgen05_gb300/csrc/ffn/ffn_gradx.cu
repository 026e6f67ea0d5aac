// dX = sum_s D_s W_s: one contraction over the pre-activation gradients of linear_act
// (one segment) or gated_ffn (two).
#include "ffn_launch.cuh"

namespace igc {

namespace {

FfnProblem sizes(const GradArgs& a) {
  FfnProblem q;
  q.M = a.M, q.N = a.K, q.K = a.N, q.dtype = a.dtype;
  q.segs = q.count_a = q.count_b = a.count;
  return q;
}

}  // namespace

int ffn_plan_x(const DeviceInfo& dev, const GradArgs& a, ProductPlan* plan) {
  FfnProblem q = sizes(a);
  for (int i = 0; i < a.count; ++i) q.A[i] = packed_rows(a.N), q.B[i] = packed_rows(a.K);
  return ffn_plan<FfnOp::GradX>(dev, q, plan);
}

int ffn_grad_x(const DeviceInfo& dev, const GradArgs& a, const ProductPlan& plan, bool late_wait,
               cudaStream_t stream) {
  FfnProblem q = sizes(a);
  for (int i = 0; i < a.count; ++i) q.A[i] = a.D[i], q.B[i] = a.W[i];
  q.out[0] = a.dX;
  q.late_wait = late_wait;
  return ffn_launch<FfnOp::GradX>(dev, q, plan, stream);
}

}  // namespace igc
