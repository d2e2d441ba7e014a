// fp32 attention over a paged cache: blocks of at most 1 heads.
#include "paged_f32.cuh"

namespace rowops {
cudaError_t paged_attention_f32_g1(const PagedArgs& a, void* workspace, const LaunchCfg& cfg) {
    return paged_f32<1>(a, workspace, cfg);
}
}  // namespace rowops
