// Group norm + activation and its backward, bf16.
#include "groupnorm_inst.cuh"

namespace rowops {
GnForwardLaunch gn_forward_bf16(int vec, int act) { return gn_forward_table<bf16_t>(vec, act); }
GnBackwardLaunch gn_backward_bf16(int vec, int act) { return gn_backward_table<bf16_t>(vec, act); }
}  // namespace rowops
