// igc_plan_ffn: the kernel and schedule that a product of the feed-forward operators runs
// with, from the launches' own decision functions, on the host.
#include "ffn_launch.cuh"

using namespace igc;

extern "C" int igc_plan_ffn(int op, int64_t M, int64_t N, int64_t K, int count, int sms,
                            int32_t* out) {
  if (out == nullptr || M <= 0 || N <= 0 || K <= 0 || sms < 2 || count < 1 || count > 2)
    return IGC_ERR_INVALID_ARG;
  if (!fits32(M) || !fits32(N) || !fits32(K)) return IGC_ERR_UNSUPPORTED;
  FfnProblem q;
  q.M = M, q.N = N, q.K = K;
  switch (op) {
    case IGC_PLAN_FFN_LINEAR: ffn_plan<FfnOp::Linear>(q, sms, out); return IGC_OK;
    case IGC_PLAN_FFN_GATED: ffn_plan<FfnOp::Gated>(q, sms, out); return IGC_OK;
    case IGC_PLAN_FFN_GRAD_X:
      q.N = K, q.K = N, q.segs = count;
      ffn_plan<FfnOp::GradX>(q, sms, out);
      return IGC_OK;
    case IGC_PLAN_FFN_GRAD_W:
      q.M = N, q.N = K, q.K = M, q.srcs = count;
      ffn_plan<FfnOp::GradW>(q, sms, out);
      return IGC_OK;
    default: return IGC_ERR_INVALID_ARG;
  }
}
