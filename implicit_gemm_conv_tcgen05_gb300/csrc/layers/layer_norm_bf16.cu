// layer_norm on bf16 rows, the residual stream in bf16.
#include "layer_norm.cuh"

namespace igc {

int layer_norm_bf16(const DeviceInfo& dev, const NormParams& p, bool drop, cudaStream_t stream) {
  return run_norm<IGC_BF16, IGC_BF16>(dev, p, drop, stream);
}

}  // namespace igc
