// groupnorm_f16.cu -- group norm kernels for f16.
#include "groupnorm_flow.cuh"
#include "groupnorm_held.cuh"

namespace rmsn {
const void *gn_flow_f16(bool backward, int chunk, int act, bool kept) { return gn_flow_t<__half>(backward, chunk, act, kept); }
const void *gn_held_f16(bool backward, int chunk, int act, bool kept) { return gn_held_t<__half>(backward, chunk, act, kept); }
}  // namespace rmsn
