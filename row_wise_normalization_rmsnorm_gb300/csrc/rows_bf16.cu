// rows_bf16.cu -- kernels on training rows (8-bit checkpoints, embedding rows) for bf16.
#include "rows_kernels.cuh"

namespace rmsn {
const void *rows_other_bf16(int which) { return rows_other_t<__nv_bfloat16>(which); }
RowKernels rows_fwd_bf16(int src, int N, bool wide) { return rows_fwd_t<__nv_bfloat16>(src, N, wide); }
RowKernels rows_bwd_bf16(bool fused, int N, bool wide) { return rows_bwd_t<__nv_bfloat16>(fused, N, wide); }
}  // namespace rmsn
