// layer_norm_backward on bf16 rows, the residual stream in bf16.
#include "layer_norm_bwd.cuh"

namespace igc {

int layer_norm_bwd_bf16(const DeviceInfo& dev, const NormBwdParams& p, bool drop, int* blocks,
                        cudaStream_t stream) {
  return run_norm_bwd<IGC_BF16, IGC_BF16>(dev, p, drop, blocks, stream);
}

}  // namespace igc
