// layer_norm on fp16 rows, the residual stream in fp16.
#include "layer_norm.cuh"

namespace igc {

int layer_norm_f16(const DeviceInfo& dev, const NormParams& p, bool drop, cudaStream_t stream) {
  return run_norm<IGC_F16, IGC_F16>(dev, p, drop, stream);
}

}  // namespace igc
