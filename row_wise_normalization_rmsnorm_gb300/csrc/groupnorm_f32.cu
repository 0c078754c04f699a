// groupnorm_f32.cu -- group norm kernels for f32.
#include "groupnorm_flow.cuh"
#include "groupnorm_held.cuh"

namespace rmsn {
const void *gn_flow_f32(bool backward, int chunk, int act, bool kept) { return gn_flow_t<float>(backward, chunk, act, kept); }
const void *gn_held_f32(bool backward, int chunk, int act, bool kept) { return gn_held_t<float>(backward, chunk, act, kept); }
}  // namespace rmsn
