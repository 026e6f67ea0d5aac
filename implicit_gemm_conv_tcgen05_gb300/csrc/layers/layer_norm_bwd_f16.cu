// layer_norm_backward on fp16 rows, the residual stream in fp16 or fp32.
#include "layer_norm_bwd.cuh"

namespace igc {

int layer_norm_bwd_f16(const DeviceInfo& dev, const NormBwdParams& p, int s_dtype, bool drop,
                     int* blocks, cudaStream_t stream) {
  return s_dtype == IGC_F32 ? run_norm_bwd<IGC_F16, IGC_F32>(dev, p, drop, blocks, stream)
                            : run_norm_bwd<IGC_F16, IGC_F16>(dev, p, drop, blocks, stream);
}

}  // namespace igc
