// layer_norm on fp32 rows.
#include "layer_norm.cuh"

namespace igc {

int layer_norm_f32(const DeviceInfo& dev, const NormParams& p, bool drop, cudaStream_t stream) {
  return run_norm<IGC_F32, IGC_F32>(dev, p, drop, stream);
}

}  // namespace igc
