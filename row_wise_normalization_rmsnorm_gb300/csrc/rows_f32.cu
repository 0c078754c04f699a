// rows_f32.cu -- kernels on training rows (8-bit checkpoints, embedding rows) for f32.
#include "rows_kernels.cuh"

namespace rmsn {
const void *rows_other_f32(int which) { return rows_other_t<float>(which); }
RowKernels rows_fwd_f32(int src, int N, bool wide) { return rows_fwd_t<float>(src, N, wide); }
RowKernels rows_bwd_f32(bool fused, int N, bool wide) { return rows_bwd_t<float>(fused, N, wide); }
}  // namespace rmsn
