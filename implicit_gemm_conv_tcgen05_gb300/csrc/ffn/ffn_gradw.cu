// dW_s = D_s^T X: the weight gradients of linear_act (one matrix) or gated_ffn (two,
// in one launch).
#include "ffn_launch.cuh"

namespace igc {

namespace {

FfnProblem sizes(const GradArgs& a) {
  FfnProblem q;
  q.M = a.N, q.N = a.K, q.K = a.M, q.dtype = a.dtype;
  q.srcs = q.count_a = a.count;
  return q;
}

}  // namespace

int ffn_plan_w(const DeviceInfo& dev, const GradArgs& a, ProductPlan* plan) {
  FfnProblem q = sizes(a);
  for (int i = 0; i < a.count; ++i) q.A[i] = packed_rows(a.N);
  q.B[0] = packed_rows(a.K);
  return ffn_plan<FfnOp::GradW>(dev, q, plan);
}

int ffn_grad_w(const DeviceInfo& dev, const GradArgs& a, const ProductPlan& plan, bool late_wait,
               cudaStream_t stream) {
  FfnProblem q = sizes(a);
  for (int i = 0; i < a.count; ++i) q.A[i] = a.D[i], q.out[i] = a.dW[i];
  q.B[0] = a.X;
  q.late_wait = late_wait;
  return ffn_launch<FfnOp::GradW>(dev, q, plan, stream);
}

}  // namespace igc
