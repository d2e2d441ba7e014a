// Group norm + activation and its backward, fp32.
#include "groupnorm_inst.cuh"

namespace rowops {
GnForwardLaunch gn_forward_f32(int vec, int act) { return gn_forward_table<float>(vec, act); }
GnBackwardLaunch gn_backward_f32(int vec, int act) { return gn_backward_table<float>(vec, act); }
}  // namespace rowops
