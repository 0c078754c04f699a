// groupnorm_f32.cu -- group norm kernels for f32.
#include "groupnorm_held.cuh"

namespace rmsn {
const void *gn_flow_f32(bool backward, bool wide, int act, bool kept) { return gn_flow_t<float>(backward, wide, act, kept); }
const void *gn_held_f32(bool backward, bool wide, int act, bool kept) { return gn_held_t<float>(backward, wide, act, kept); }
}  // namespace rmsn
