// bf16 instantiations of RMSNorm with an 8-bit result.
#include "norm_quant.cuh"

namespace rowops {
cudaError_t rms_quant_bf16(const QuantArgs& a, int piece, const LaunchCfg& cfg) {
    return launch_rms_quant<bf16_t>(a, piece, cfg);
}
}  // namespace rowops
