// igc_plan_ffn: the kernel and schedule that a product of the feed-forward operators runs
// with, from the launches' own decision functions, on the host.
#include "ffn_launch.cuh"

using namespace igc;

namespace {

// igc_plan_ffn's answer, or (res) what a CTA of its kernel takes.
template <FfnOp kOp>
void plan_out(const FfnProblem& q, const ProductPlan& p, int32_t* out, bool res) {
  if (res)
    ffn_resources_host<kOp>(q, p, out);
  else
    ffn_plan_out(q, p, out);
}

int plan_host(int op, int64_t M, int64_t N, int64_t K, int count, int sms, int32_t* out,
              bool res) {
  if (out == nullptr || M <= 0 || N <= 0 || K <= 0 || sms < 2 || count < 1 || count > 2)
    return IGC_ERR_INVALID_ARG;
  if (!fits32(M) || !fits32(N) || !fits32(K)) return IGC_ERR_UNSUPPORTED;
  FfnProblem q;
  q.M = M, q.N = N, q.K = K;
  const FfnProblem qx = grad_x_problem(M, N, K, IGC_BF16, count);
  const FfnProblem qw = grad_w_problem(M, N, K, IGC_BF16, count);
  switch (op) {
    case IGC_PLAN_FFN_LINEAR:
      plan_out<FfnOp::Linear>(q, ffn_plan_host<FfnOp::Linear>(q, sms), out, res);
      return IGC_OK;
    case IGC_PLAN_FFN_GATED:
      plan_out<FfnOp::Gated>(q, ffn_plan_host<FfnOp::Gated>(q, sms), out, res);
      return IGC_OK;
    case IGC_PLAN_FFN_GRAD_X: {
      ProductPlan p = ffn_plan_host<FfnOp::GradX>(qx, sms);
      if (grad_x_beside_w(p, ffn_plan_host<FfnOp::GradW>(qw, sms), sms)) p.small = false;
      plan_out<FfnOp::GradX>(qx, p, out, res);
      return IGC_OK;
    }
    case IGC_PLAN_FFN_GRAD_W:
      plan_out<FfnOp::GradW>(qw, ffn_plan_host<FfnOp::GradW>(qw, sms), out, res);
      return IGC_OK;
    default: return IGC_ERR_INVALID_ARG;
  }
}

}  // namespace

extern "C" int igc_plan_ffn(int op, int64_t M, int64_t N, int64_t K, int count, int sms,
                            int32_t* out) {
  return plan_host(op, M, N, K, count, sms, out, false);
}

extern "C" int igc_ffn_cta_resources(int op, int64_t M, int64_t N, int64_t K, int count, int sms,
                                     int32_t* out) {
  return plan_host(op, M, N, K, count, sms, out, true);
}
