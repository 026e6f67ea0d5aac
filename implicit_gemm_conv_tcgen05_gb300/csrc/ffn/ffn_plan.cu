// Tensor maps of the feed-forward launches, and igc_plan_ffn: the kernel and schedule that
// a product of the feed-forward operators runs with, from the launches' own decision
// functions, on the host.
#include "ffn_launch.cuh"

namespace igc {

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled through the runtime (the library does not link libcuda).
EncodeTiledFn encoder() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

}  // namespace

int encode_tiled_2d_fresh(CUtensorMap* map, CUtensorMapDataType dtype, const void* base,
                          uint64_t inner, uint64_t rows, uint64_t row_stride_bytes,
                          uint32_t box_inner, uint32_t box_rows) {
  const EncodeTiledFn encode = encoder();
  if (encode == nullptr) return IGC_ERR_CUDA;
  const cuuint64_t dims[2] = {inner, rows};
  const cuuint64_t strides[1] = {row_stride_bytes};
  const cuuint32_t box[2] = {box_inner, box_rows};
  const cuuint32_t steps[2] = {1, 1};
  return encode(map, dtype, 2, const_cast<void*>(base), dims, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? IGC_OK
             : IGC_ERR_CUDA;
}

}  // namespace igc

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
