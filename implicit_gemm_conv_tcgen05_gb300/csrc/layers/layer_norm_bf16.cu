// layer_norm on bf16 rows, the residual stream in bf16 or fp32.
#include "layer_norm.cuh"

namespace igc {

int layer_norm_bf16(const DeviceInfo& dev, const NormParams& p, int s_dtype, bool drop,
                    cudaStream_t stream) {
  return s_dtype == IGC_F32 ? run_norm<IGC_BF16, IGC_F32>(dev, p, drop, stream)
                            : run_norm<IGC_BF16, IGC_BF16>(dev, p, drop, stream);
}

}  // namespace igc
