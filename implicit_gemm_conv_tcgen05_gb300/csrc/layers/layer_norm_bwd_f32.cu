// layer_norm_backward on fp32 rows.
#include "layer_norm_bwd.cuh"

namespace igc {

int layer_norm_bwd_f32(const DeviceInfo& dev, const NormBwdParams& p, bool drop, int* blocks,
                       cudaStream_t stream) {
  return run_norm_bwd<IGC_F32, IGC_F32>(dev, p, drop, blocks, stream);
}

}  // namespace igc
