// train_rows.h -- host helpers shared by the entry points on training rows
// (group norm, 8-bit checkpoints, embedding rows).
#pragma once

#include <initializer_list>
#include <utility>

#include "common.cuh"
#include "head_rows.h"
#include "plans.h"

namespace rmsn {

// A launch as a programmatic dependent; a cudaError_t.
inline int launch(const void *k, unsigned x, unsigned y, int threads, size_t smem, void **args, cudaStream_t s, unsigned cluster = 0) {
    if (smem > 48 * 1024) {
        const int e = allow_staged_smem(k);
        if (e != 0) return e;
    }
    LaunchCfg lc(x, (unsigned)threads, smem, s, cluster);
    lc.cfg.gridDim.y = y;
    return (int)cudaLaunchKernelExC(&lc.cfg, k, args);
}

// Zeros for what a sum over nothing gives.
inline rmsnorm_status_t zeros(std::initializer_list<std::pair<void *, size_t>> out, cudaStream_t s) {
    for (const auto &o : out)
        if (o.first && o.second) {
            const cudaError_t e = cudaMemsetAsync(o.first, 0, o.second, s);
            if (e != cudaSuccess) return head_cuda_fail((int)e);
        }
    return RMSNORM_SUCCESS;
}

// `run` on the caller's workspace (at least `need` bytes on a 16-byte
// boundary), or on stream-ordered memory.
template <class F>
rmsnorm_status_t with_workspace(void *workspace, size_t have, size_t need, cudaStream_t s, F &&run) {
    if (workspace) {
        if (!on(workspace, 16) || have < need) return RMSNORM_ERR_WORKSPACE;
        return run(static_cast<char *>(workspace));
    }
    void *tmp = nullptr;
    cudaError_t e = cudaMallocAsync(&tmp, need, s);
    if (e != cudaSuccess) return head_cuda_fail((int)e);
    const rmsnorm_status_t st = run(static_cast<char *>(tmp));
    e = cudaFreeAsync(tmp, s);
    return st != RMSNORM_SUCCESS || e == cudaSuccess ? st : head_cuda_fail((int)e);
}

inline int base_of(int dt) { return dt & ~RMSNORM_WEIGHT_F32; }
inline bool known_dtype(int dt) {
    const int b = base_of(dt);
    return b == RMSNORM_F32 || b == RMSNORM_BF16 || b == RMSNORM_F16;
}
inline int bytes_of(int dt) { return base_of(dt) == RMSNORM_F32 ? 4 : 2; }
inline int weight_bytes(int dt) { return (dt & RMSNORM_WEIGHT_F32) ? 4 : bytes_of(dt); }

}  // namespace rmsn
