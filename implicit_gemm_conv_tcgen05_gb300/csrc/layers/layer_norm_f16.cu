// layer_norm on fp16 rows, the residual stream in fp16 or fp32.
#include "layer_norm.cuh"

namespace igc {

int layer_norm_f16(const DeviceInfo& dev, const NormParams& p, int s_dtype, bool drop,
                   cudaStream_t stream) {
  return s_dtype == IGC_F32 ? run_norm<IGC_F16, IGC_F32>(dev, p, drop, stream)
                            : run_norm<IGC_F16, IGC_F16>(dev, p, drop, stream);
}

}  // namespace igc
