// layer_norm on bf16 rows, the residual stream in fp32.
#include "layer_norm.cuh"

namespace igc {

int layer_norm_bf16_f32(const DeviceInfo& dev, const NormParams& p, bool drop,
                        cudaStream_t stream) {
  return run_norm<IGC_BF16, IGC_F32>(dev, p, drop, stream);
}

}  // namespace igc
