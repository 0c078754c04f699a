// rows_f16.cu -- kernels on training rows (8-bit checkpoints, embedding rows) for f16.
#include "rows_kernels.cuh"

namespace rmsn {
const void *rows_other_f16(int which) { return rows_other_t<__half>(which); }
RowKernels rows_fwd_f16(int src, int N, bool wide) { return rows_fwd_t<__half>(src, N, wide); }
RowKernels rows_bwd_f16(bool fused, int N, bool wide) { return rows_bwd_t<__half>(fused, N, wide); }
}  // namespace rmsn
