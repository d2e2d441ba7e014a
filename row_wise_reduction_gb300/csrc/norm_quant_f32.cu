// fp32 instantiations of RMSNorm with an 8-bit result.
#include "norm_quant.cuh"

namespace rowops {
cudaError_t rms_quant_f32(const QuantArgs& a, int piece, const LaunchCfg& cfg) { return launch_rms_quant<float>(a, piece, cfg); }
}  // namespace rowops
