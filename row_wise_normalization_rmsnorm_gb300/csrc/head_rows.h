// head_rows.h -- host helpers shared by the entry points on head rows
// (rotary positions, the paged cache, its attention).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/rmsnorm.h"

namespace rmsn {

void set_last_cuda_error(int e);                // api.cu
// api.cu: cudaError_t; status and dev may be NULL
int current_device(int *sms, int **status, int *dev = nullptr);
int allow_staged_smem(const void *k);           // api.cu: cudaError_t

inline rmsnorm_status_t head_cuda_fail(int e) {
    set_last_cuda_error(e);
    return RMSNORM_ERR_CUDA;
}

inline bool on(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

// A stride counts only where its dimension has more than one entry.
inline int64_t stride_of(int64_t stride, int64_t entries) { return entries > 1 ? stride : 0; }

// False where a written dimension's entries would share their place: the rows
// would overwrite one another in no order.
inline bool apart(int64_t stride, int64_t entries) { return entries <= 1 || stride != 0; }

}  // namespace rmsn
