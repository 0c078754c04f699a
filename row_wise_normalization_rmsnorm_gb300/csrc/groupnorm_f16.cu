// groupnorm_f16.cu -- group norm kernels for f16.
#include "groupnorm_held.cuh"

namespace rmsn {
const void *gn_flow_f16(bool backward, bool wide, int act, bool kept) { return gn_flow_t<__half>(backward, wide, act, kept); }
const void *gn_held_f16(bool backward, bool wide, int act, bool kept) { return gn_held_t<__half>(backward, wide, act, kept); }
}  // namespace rmsn
