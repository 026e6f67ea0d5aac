// layer_norm_backward on bf16 rows, the residual stream in bf16 or fp32.
#include "layer_norm_bwd.cuh"

namespace igc {

int layer_norm_bwd_bf16(const DeviceInfo& dev, const NormBwdParams& p, int s_dtype, bool drop,
                     int* blocks, cudaStream_t stream) {
  return s_dtype == IGC_F32 ? run_norm_bwd<IGC_BF16, IGC_F32>(dev, p, drop, blocks, stream)
                            : run_norm_bwd<IGC_BF16, IGC_BF16>(dev, p, drop, blocks, stream);
}

}  // namespace igc
