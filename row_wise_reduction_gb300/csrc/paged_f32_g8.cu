// fp32 attention over a paged cache: blocks of at most 8 heads.
#include "paged_f32.cuh"

namespace rowops {
cudaError_t paged_attention_f32_g8(const PagedArgs& a, void* workspace, const LaunchCfg& cfg) {
    return paged_f32<8>(a, workspace, cfg);
}
}  // namespace rowops
