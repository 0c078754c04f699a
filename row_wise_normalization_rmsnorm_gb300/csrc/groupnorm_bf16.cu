// groupnorm_bf16.cu -- group norm kernels for bf16.
#include "groupnorm_flow.cuh"
#include "groupnorm_held.cuh"

namespace rmsn {
const void *gn_flow_bf16(bool backward, int chunk, int act, bool kept) { return gn_flow_t<__nv_bfloat16>(backward, chunk, act, kept); }
const void *gn_held_bf16(bool backward, int chunk, int act, bool kept) { return gn_held_t<__nv_bfloat16>(backward, chunk, act, kept); }
}  // namespace rmsn
