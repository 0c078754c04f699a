// rows_kernels.cuh -- RMSNorm forward from other rows than an activation
// matrix's (embedding rows) and with its input kept in 8 bits, the backward
// that reads what was kept, and keeping and restoring rows by themselves.
//
//   forward   h = x, R(x + residual) or R(scale table[id]),  y and rstd of h as rmsnorm_fwd
//             codes, scales: h in 8 bits (rows8.cuh)
//   backward  xhat = rstd value(code), the rest as rmsnorm_bwd:
//             g = dy (offset + w),  c = (1/N) sum g xhat,  dx = rstd (g - xhat c) [+ dres],  dw = sum dy xhat
//
// All of it is bound by memory: bytes a value of bf16 are 5.03 for the
// forward with its checkpoint (x, y, code), 5.03 for the backward. 16384 x 8192
// in bf16, each by itself: 105 us (6.4 TB/s) and 129 us (5.3), of 101 at the rate
// of a copy; one after the other 236.
#pragma once

#include "rows8.cuh"

namespace rmsn {

enum { kSrcPlain = 0, kSrcAdd = 1, kSrcEmbed = 2 };

struct RowsParams {
    const void *x, *residual, *w;  // x: the table for kSrcEmbed
    const void *ids;               // kSrcEmbed: int32 or int64 [M]
    void *y, *h;                   // y NULL: the rows alone (kSrcEmbed)
    float *rstd;
    uint8_t *codes, *scales;
    int64_t vocab;
    int M, N, id_bytes, w32;
    float scale, eps, offset;
};

struct RowsBwdParams {
    const void *dy, *dres, *w;
    const uint8_t *codes, *scales;
    const float *rstd;
    void *dx;
    float *ws;  // [gridDim.x, N] partial dw, NULL without w
    int M, N, w32;
    int stage_rows, depth;  // rows a stage holds, stages
    float offset;
    int *status;
};

// The table row of token `row` (NULL: none, the id is outside the table).
template <typename T> __device__ __forceinline__ const T *table_row(const RowsParams &p, int64_t row) {
    const int64_t id = p.id_bytes == 8 ? static_cast<const int64_t *>(p.ids)[row] : (int64_t) static_cast<const int32_t *>(p.ids)[row];
    return id >= 0 && id < p.vocab ? static_cast<const T *>(p.x) + id * p.N : nullptr;
}

template <typename T>
__device__ __forceinline__ void weights_at(const void *w, int w32, int c, float offset, float2 (&f)[Elem<T>::NP]) {
    if (!w) {
#pragma unroll
        for (int q = 0; q < Elem<T>::NP; ++q) f[q] = make_float2(1.f, 1.f);
        return;
    }
    if (w32)
        load_w_chunk<T, float>(w, c, f);
    else
        load_w_chunk<T, T>(w, c, f);
#pragma unroll
    for (int q = 0; q < Elem<T>::NP; ++q) f[q] = make_float2(offset + f[q].x, offset + f[q].y);
}

__device__ __forceinline__ float rstd_of(float ss, int N, float eps) { return 1.f / sqrtf(ss / (float)N + eps); }

// ----------------------------------------------------------------- forward --
// A team of TPR threads a row, the row in registers (V 16-byte chunks a
// thread), read once.
template <typename T, int TPR, int V, int SRC, bool KEEP>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256) rows_fwd(const RowsParams p) {
    constexpr int E = Elem<T>::E, NP = Elem<T>::NP, TEAMS = TPR >= 256 ? 1 : 256 / TPR, W = TPR > 32 ? TPR / 32 : 1;
    __shared__ float red[TEAMS][W];
    pdl_wait();
    pdl_trigger();
    const int team = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * TEAMS + team;
    const bool ok = row < p.M;
    const int C = p.N / E;
    const uint4 *src = nullptr;
    if (ok) {
        if constexpr (SRC == kSrcEmbed)
            src = reinterpret_cast<const uint4 *>(table_row<T>(p, row));
        else
            src = static_cast<const uint4 *>(p.x) + row * C;
    }
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 h[V], r[SRC == kSrcAdd ? V : 1];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = v * TPR + t;
        const bool in = src && c < C;
        // a table row may be another token's too: the other rows are read once
        h[v] = !in ? zero : SRC == kSrcEmbed ? src[c] : ld_stream(src + c);
        if constexpr (SRC == kSrcAdd) r[v] = in ? ld_stream(static_cast<const uint4 *>(p.residual) + row * C + c) : zero;
    }
    float2 ss = make_float2(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = v * TPR + t;
        float2 a[NP];
        unpack<T>(h[v], a);
        if constexpr (SRC != kSrcPlain) {
            if constexpr (SRC == kSrcAdd) {
                float2 b[NP];
                unpack<T>(r[v], b);
#pragma unroll
                for (int q = 0; q < NP; ++q) a[q] = Pair<true>::add(a[q], b[q]);
            } else {
#pragma unroll
                for (int q = 0; q < NP; ++q) a[q] = Pair<true>::mul(a[q], make_float2(p.scale, p.scale));
            }
            h[v] = pack<T>(a);
            if (ok && c < C) static_cast<uint4 *>(p.h)[row * C + c] = h[v];
            unpack<T>(h[v], a);  // as stored
        }
#pragma unroll
        for (int q = 0; q < NP; ++q) ss = Pair<true>::fma(a[q], a[q], ss);
    }
    const float rstd = rstd_of(team_allreduce<TPR>(ss.x + ss.y, red[team], t), p.N, p.eps);
    if (ok && t == 0) p.rstd[row] = rstd;
    const int64_t blocks = (p.N + kBlock8 - 1) / kBlock8;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = v * TPR + t;
        const bool in = ok && c < C;
        float2 a[NP];
        unpack<T>(h[v], a);
        if constexpr (KEEP)
            keep_chunk<T>(h[v], in, 0xffffffffu, p.codes + row * p.N + c * E, p.scales + row * blocks + c * E / kBlock8);
        if (in) {
            float2 f[NP];
            weights_at<T>(p.w, p.w32, c, p.offset, f);
#pragma unroll
            for (int q = 0; q < NP; ++q) a[q] = Pair<true>::mul(Pair<true>::mul(a[q], make_float2(rstd, rstd)), f[q]);
            static_cast<uint4 *>(p.y)[row * C + c] = pack<T>(a);
        }
    }
}

// Rows of any alignment, value by value: a team of TPR threads (whole warps) a
// row, K values a thread in registers, all loads under way at once. Consecutive
// lanes take consecutive values, so a warp's 32 are a block.
template <typename T, int TPR, int K, int SRC, bool KEEP>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256) rows_fwd_lanes(const RowsParams p) {
    constexpr int TEAMS = TPR >= 256 ? 1 : 256 / TPR, W = TPR / 32;
    __shared__ float red[TEAMS][W];
    pdl_wait();
    pdl_trigger();
    const int team = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * TEAMS + team;
    const bool ok = row < p.M;
    const T *src = nullptr;
    if (ok) {
        if constexpr (SRC == kSrcEmbed)
            src = table_row<T>(p, row);
        else
            src = static_cast<const T *>(p.x) + row * p.N;
    }
    float v[K], r[SRC == kSrcAdd ? K : 1];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int j = k * TPR + t;
        v[k] = src && j < p.N ? load_elem(src, j) : 0.f;
        if constexpr (SRC == kSrcAdd) r[k] = src && j < p.N ? load_elem(static_cast<const T *>(p.residual) + row * p.N, j) : 0.f;
    }
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int j = k * TPR + t;
        if constexpr (SRC != kSrcPlain) {
            v[k] = round_to(SRC == kSrcAdd ? v[k] + r[k] : v[k] * p.scale, static_cast<const T *>(nullptr));
            if (ok && j < p.N) store_elem(static_cast<T *>(p.h) + row * p.N, j, v[k]);
        }
        ss = fmaf(v[k], v[k], ss);
    }
    if constexpr (SRC == kSrcEmbed) {
        if (!p.y) return;
    }
    const float rstd = rstd_of(team_allreduce<TPR>(ss, red[team], t), p.N, p.eps);
    if (ok && t == 0) p.rstd[row] = rstd;
    const int blocks = (p.N + kBlock8 - 1) / kBlock8;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int j = k * TPR + t;
        const bool in = ok && j < p.N;
        if constexpr (KEEP) {
            const uint32_t b = scale8<T>(__reduce_max_sync(0xffffffffu, abs_bits(v[k])));
            if (in) p.codes[row * p.N + j] = code8(v[k], b);
            if (in && (t & 31) == 0) p.scales[row * blocks + j / kBlock8] = (uint8_t)b;
        }
        if (in) {
            const float f = !p.w ? 1.f : p.offset + (p.w32 ? load_w(static_cast<const float *>(p.w), j) : load_w(static_cast<const T *>(p.w), j));
            store_elem(static_cast<T *>(p.y) + row * p.N, j, v[k] * rstd * f);
        }
    }
}

// The same for rows of any length: a CTA a row, read twice.
template <typename T, int SRC, bool KEEP>
__global__ void __launch_bounds__(256) rows_fwd_any(const RowsParams p) {
    __shared__ float red[32];
    pdl_wait();
    pdl_trigger();
    const int64_t row = blockIdx.x;
    const T *src;
    if constexpr (SRC == kSrcEmbed)
        src = table_row<T>(p, row);
    else
        src = static_cast<const T *>(p.x) + row * p.N;
    T *h = SRC == kSrcPlain ? nullptr : static_cast<T *>(p.h) + row * p.N;
    const T *res = static_cast<const T *>(p.residual) + row * p.N;
    float ss = 0.f;
    for (int j = threadIdx.x; j < p.N; j += 256) {
        float v = src ? load_elem(src, j) : 0.f;
        if constexpr (SRC == kSrcAdd) v = v + load_elem(res, j);
        if constexpr (SRC == kSrcEmbed) v = v * p.scale;
        if constexpr (SRC != kSrcPlain) {
            store_elem(h, j, v);
            v = round_to(v, h);
        }
        ss = fmaf(v, v, ss);
    }
    if constexpr (SRC == kSrcEmbed) {
        if (!p.y) return;
    }
    const float rstd = rstd_of(cta_allreduce(ss, red), p.N, p.eps);
    if (threadIdx.x == 0) p.rstd[row] = rstd;
    T *y = static_cast<T *>(p.y) + row * p.N;
    const int blocks = (p.N + kBlock8 - 1) / kBlock8;
    for (int j0 = threadIdx.x & ~31; j0 < p.N; j0 += 256) {
        const int j = j0 + (threadIdx.x & 31);
        const bool in = j < p.N;
        // h is this thread's own store of above
        const float v = !in ? 0.f : SRC == kSrcPlain ? load_elem(src, j) : load_elem(h, j);
        if constexpr (KEEP) {
            const uint32_t b = scale8<T>(__reduce_max_sync(0xffffffffu, abs_bits(v)));
            if (in) p.codes[row * p.N + j] = code8(v, b);
            if ((threadIdx.x & 31) == 0) p.scales[row * blocks + j0 / kBlock8] = (uint8_t)b;
        }
        if (in) {
            const float f = !p.w ? 1.f : p.offset + (p.w32 ? load_w(static_cast<const float *>(p.w), j) : load_w(static_cast<const T *>(p.w), j));
            store_elem(y, j, v * rstd * f);
        }
    }
}

// Embedding rows alone, 16-byte chunks: a warp takes 32 V neighbouring chunks of a row.
template <typename T, int V>
__global__ void __launch_bounds__(256) embed_rows(const RowsParams p, int tiles) {
    constexpr int NP = Elem<T>::NP;
    pdl_wait();
    pdl_trigger();
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t row = item / tiles;
    if (row >= p.M) return;
    const int C = p.N / Elem<T>::E, c0 = (int)(item - row * tiles) * 32 * V + (threadIdx.x & 31);
    const uint4 *src = reinterpret_cast<const uint4 *>(table_row<T>(p, row));
    uint4 h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = src && c0 + 32 * v < C ? src[c0 + 32 * v] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (c0 + 32 * v < C) {
            float2 a[NP];
            unpack<T>(h[v], a);
#pragma unroll
            for (int q = 0; q < NP; ++q) a[q] = Pair<true>::mul(a[q], make_float2(p.scale, p.scale));
            static_cast<uint4 *>(p.h)[row * C + c0 + 32 * v] = pack<T>(a);
        }
}

// -------------------------------------------------------- keep and restore --
// Whole blocks (N % 32 == 0): the matrix is one row of blocks. Chunks of 16
// bytes, V of them a thread in flight.
constexpr int kPackChunks = 4;
template <typename T>
__global__ void __launch_bounds__(256) pack_blocks(const uint4 *x, uint8_t *codes, uint8_t *scales, int64_t chunks) {
    constexpr int E = Elem<T>::E;
    pdl_wait();
    pdl_trigger();
    const int64_t c0 = (int64_t)blockIdx.x * 256 * kPackChunks + threadIdx.x;
    uint4 r[kPackChunks];
#pragma unroll
    for (int k = 0; k < kPackChunks; ++k) r[k] = c0 + 256 * k < chunks ? ld_stream(x + c0 + 256 * k) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < kPackChunks; ++k) {
        const int64_t c = c0 + 256 * k;
        keep_chunk<T>(r[k], c < chunks, 0xffffffffu, codes + c * E, scales + c * E / kBlock8);
    }
}

// A restored value: never an infinity where the value was finite (64 steps of
// the largest scale are finite).
template <typename T>
__global__ void __launch_bounds__(256) unpack_blocks(const uint8_t *codes, const uint8_t *scales, uint4 *x, int64_t chunks) {
    constexpr int E = Elem<T>::E, NP = Elem<T>::NP;
    using W = typename std::conditional<E == 8, uint2, uint32_t>::type;
    pdl_wait();
    pdl_trigger();
    const int64_t c0 = (int64_t)blockIdx.x * 256 * kPackChunks + threadIdx.x;
    W r[kPackChunks];
    uint32_t b[kPackChunks];
#pragma unroll
    for (int k = 0; k < kPackChunks; ++k) {
        const int64_t c = c0 + 256 * k;
        if (c < chunks) {
            r[k] = __ldcs(reinterpret_cast<const W *>(codes) + c);
            b[k] = scales[c * E / kBlock8];
        }
    }
#pragma unroll
    for (int k = 0; k < kPackChunks; ++k)
        if (c0 + 256 * k < chunks) {
            const float f = from_codes8(b[k]);
            float2 a[NP];
#pragma unroll
            for (int i = 0; i < E / 4; ++i) {
                float d[4];
                uint32_t w;
                if constexpr (E == 8)
                    w = i ? r[k].y : r[k].x;
                else
                    w = r[k];
                decode8x4(w, d);
                a[2 * i] = make_float2(d[0] * f, d[1] * f);
                a[2 * i + 1] = make_float2(d[2] * f, d[3] * f);
            }
            x[c0 + 256 * k] = pack<T>(a);
        }
}

// Rows of any length and alignment: a warp takes a run of kRun neighbouring
// blocks of a row, a value a lane.
constexpr int kRun = 8;
struct Run {
    int64_t row;
    int block, n;  // first block, blocks
    __device__ __forceinline__ Run(int64_t M, int blocks) {
        const int runs = (blocks + kRun - 1) / kRun;
        const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
        row = item / runs;
        block = (int)(item - row * runs) * kRun;
        n = row < M ? min(kRun, blocks - block) : 0;
    }
};
// A run's blocks: FULL, all kRun of them whole (no test a value).
template <typename T, bool FULL>
__device__ __forceinline__ void pack_run(const T *src, uint8_t *dst, int left, uint32_t &mine) {
    const int lane = threadIdx.x & 31;
    float v[kRun];
#pragma unroll
    for (int k = 0; k < kRun; ++k) v[k] = FULL || k * kBlock8 < left ? load_elem(src, k * kBlock8) : 0.f;
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
        const uint32_t b = scale8<T>(__reduce_max_sync(0xffffffffu, abs_bits(v[k])));
        if (FULL || k * kBlock8 < left) dst[k * kBlock8] = code8(v[k], b);
        if (lane == k) mine = b;
    }
}
template <typename T>
__global__ void __launch_bounds__(256) pack_any(const T *x, uint8_t *codes, uint8_t *scales, int64_t M, int N) {
    pdl_wait();
    pdl_trigger();
    const int blocks = (N + kBlock8 - 1) / kBlock8, lane = threadIdx.x & 31;
    const Run run(M, blocks);
    const int j0 = run.block * kBlock8 + lane;
    const T *src = x + run.row * N + j0;
    uint8_t *dst = codes + run.row * N + j0;
    uint32_t mine = 0;
    if (run.n == kRun && (run.block + kRun) * kBlock8 <= N)  // (the same in the whole warp)
        pack_run<T, true>(src, dst, 0, mine);
    else
        pack_run<T, false>(src, dst, run.n > 0 ? N - j0 : 0, mine);
    if (lane < run.n) scales[run.row * blocks + run.block + lane] = (uint8_t)mine;
}

template <typename T, bool FULL>
__device__ __forceinline__ void unpack_run(const uint8_t *src, T *dst, int left, float f) {
    uint8_t c[kRun];
#pragma unroll
    for (int k = 0; k < kRun; ++k) c[k] = FULL || k * kBlock8 < left ? src[k * kBlock8] : (uint8_t)0;
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
        const float fk = __shfl_sync(0xffffffffu, f, k);
        // (as decode8x4)
        const float v = __uint_as_float(((uint32_t)c[k] ^ 0x80u) | 0x4b000000u) - 8388736.f;
        if (FULL || k * kBlock8 < left) store_elem(dst, k * kBlock8, v * fk);
    }
}
template <typename T>
__global__ void __launch_bounds__(256) unpack_any(const uint8_t *codes, const uint8_t *scales, T *x, int64_t M, int N) {
    pdl_wait();
    pdl_trigger();
    const int blocks = (N + kBlock8 - 1) / kBlock8, lane = threadIdx.x & 31;
    const Run run(M, blocks);
    const int j0 = run.block * kBlock8 + lane;
    const uint8_t *src = codes + run.row * N + j0;
    T *dst = x + run.row * N + j0;
    const float f = lane < run.n ? from_codes8(scales[run.row * blocks + run.block + lane]) : 0.f;
    if (run.n == kRun && (run.block + kRun) * kBlock8 <= N)
        unpack_run<T, true>(src, dst, 0, f);
    else
        unpack_run<T, false>(src, dst, run.n > 0 ? N - j0 : 0, f);
}

__device__ __forceinline__ uint2 lds64(const void *p) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(smem_u32(p)));
    return v;
}
__device__ __forceinline__ uint32_t lds32(const void *p) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(smem_u32(p)));
    return v;
}
__device__ __forceinline__ uint32_t lds8(const void *p) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(smem_u32(p)));
    return v;
}

// ---------------------------------------------------------------- backward --
// Persistent: CTA i takes blocks of `stage_rows` rows i, i + grid, ... A warp
// of its own keeps `depth` blocks under way into shared memory (bulk copies;
// codes and scales of a block start anywhere: the 16-byte blocks that hold
// them are copied). A team of TPR threads takes R rows at once, so that one
// barrier and one round of shuffles serve them all, reads them a second time
// from shared memory for dx, and keeps dw's sums of its columns in registers
// until the end.
__host__ __device__ constexpr uint32_t up16(uint32_t n) { return (n + 15u) & ~15u; }

struct StageLayout {  // byte offsets in a stage
    uint32_t dres, codes, scales, bytes;
    __host__ __device__ StageLayout(int rows, int N, int es, bool fused) {
        const uint32_t row = (uint32_t)rows * N, blocks = (uint32_t)rows * ((N + kBlock8 - 1) / kBlock8);
        dres = row * es;
        codes = dres + (fused ? row * es : 0u);
        scales = codes + up16(row + 15u);
        bytes = scales + up16(blocks + 15u);
    }
};

constexpr uint32_t kStageWaitLimit = 1u << 20;  // polls of a stage's copies (each may suspend the thread for a while)
constexpr int kStagesMost = 8;

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Barrier over the first N threads of the CTA.
template <int N> __device__ __forceinline__ void sync_first() { asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory"); }

__host__ __device__ constexpr int bwd_consumers(int tpr) { return tpr > 256 ? tpr : 256; }

template <typename T, int TPR, int V, int R, bool FUSED>
__global__ void __launch_bounds__(bwd_consumers(TPR) + 32, TPR > 256 ? 1 : 2) rows_bwd(const RowsBwdParams p) {
    constexpr int E = Elem<T>::E, NP = Elem<T>::NP, NT = bwd_consumers(TPR), TEAMS = NT / TPR, W = TPR > 32 ? TPR / 32 : 1;
    extern __shared__ __align__(128) uint8_t stages[];
    __shared__ float red[2][R][TEAMS][W];
    __shared__ __align__(8) uint64_t full[kStagesMost], empty[kStagesMost];
    const int C = p.N / E, nb = (p.N + kBlock8 - 1) / kBlock8;
    const StageLayout lay(p.stage_rows, p.N, sizeof(T), FUSED);
    const int blocks = (p.M + p.stage_rows - 1) / p.stage_rows;
    const int mine = blocks > (int)blockIdx.x ? (blocks - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.depth; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], NT / 32);
        }
        mbar_init_fence();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    bool failed = false;
    if (threadIdx.x >= NT) {  // the copying warp
        if (threadIdx.x == NT) {
            int stage = 0;
            uint32_t phase = 1;  // (the first wait on an unused stage returns at once)
            int64_t r0 = (int64_t)blockIdx.x * p.stage_rows;
            const int64_t step = (int64_t)gridDim.x * p.stage_rows;
            for (int i = 0; i < mine && !failed; ++i, r0 += step) {
                if (!mbar_wait(&empty[stage], phase, kStageWaitLimit)) failed = true;
                if (i >= p.depth) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                uint8_t *s = stages + (size_t)stage * lay.bytes;
                const uint32_t rows = (uint32_t)min((int64_t)p.stage_rows, p.M - r0), bytes = rows * (uint32_t)p.N * sizeof(T);
                const Cover cc = cover16(p.codes + r0 * p.N, rows * p.N), cs = cover16(p.scales + r0 * nb, rows * nb);
                mbar_arrive_expect_tx(&full[stage], bytes * (FUSED ? 2 : 1) + cc.bytes + cs.bytes);
                bulk_g2s(s, static_cast<const T *>(p.dy) + r0 * p.N, bytes, &full[stage]);
                if (FUSED) bulk_g2s(s + lay.dres, static_cast<const T *>(p.dres) + r0 * p.N, bytes, &full[stage]);
                bulk_g2s(s + lay.codes, cc.src, cc.bytes, &full[stage]);
                bulk_g2s(s + lay.scales, cs.src, cs.bytes, &full[stage]);
                if (++stage == p.depth) stage = 0, phase ^= 1u;
            }
            // (every copy is waited for by the threads that read it)
            if (failed && p.status) *p.status = 1;
        }
        return;
    }
    const int team = threadIdx.x / TPR, t = threadIdx.x % TPR;
    float2 f[V][NP], dw[V][NP];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = v * TPR + t;
#pragma unroll
        for (int q = 0; q < NP; ++q) f[v][q] = dw[v][q] = make_float2(0.f, 0.f);
        if (c < C) weights_at<T>(p.w, p.w32, c, p.offset, f[v]);
    }
    // dy and xhat of chunk c of row lr of the stage
    auto values = [&](const uint8_t *s, uint32_t oc, uint32_t os, int lr, int c, float rstd, float2 (&d)[NP], float2 (&xh)[NP]) {
        const uint32_t at = (uint32_t)lr * C + c;
        unpack<T>(lds128(s + (size_t)at * 16), d);
        const float to = rstd * from_codes8(lds8(s + lay.scales + os + lr * nb + c * E / kBlock8));
        const float2 to2 = make_float2(to, to);
        float x[4];
        if constexpr (E == 8) {
            const uint2 code = lds64(s + lay.codes + oc + at * E);
            decode8x4(code.x, x);
            xh[0] = Pair<true>::mul(make_float2(x[0], x[1]), to2);
            xh[1] = Pair<true>::mul(make_float2(x[2], x[3]), to2);
            decode8x4(code.y, x);
            xh[2] = Pair<true>::mul(make_float2(x[0], x[1]), to2);
            xh[3] = Pair<true>::mul(make_float2(x[2], x[3]), to2);
        } else {
            decode8x4(lds32(s + lay.codes + oc + at * E), x);
            xh[0] = Pair<true>::mul(make_float2(x[0], x[1]), to2);
            xh[1] = Pair<true>::mul(make_float2(x[2], x[3]), to2);
        }
    };
    const float minus_inv = -1.f / (float)p.N;
    int flip = 0, stage = 0;
    uint32_t phase = 0;
    int64_t r0 = (int64_t)blockIdx.x * p.stage_rows;
    const int64_t step = (int64_t)gridDim.x * p.stage_rows;
    for (int i = 0; i < mine; ++i, r0 += step) {
        const uint8_t *s = stages + (size_t)stage * lay.bytes;
        const uint32_t oc = addr_mod16(p.codes + r0 * p.N), os = addr_mod16(p.scales + r0 * nb);
        const int rows = (int)min((int64_t)p.stage_rows, p.M - r0);
        for (int k = 0; k < p.stage_rows; k += TEAMS * R, flip ^= 1) {
            float rstd[R], part[R];
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const int lr = k + j * TEAMS + team;
                rstd[j] = lr < rows ? p.rstd[r0 + lr] : 0.f;
            }
            if (k == 0 && !failed && !mbar_wait(&full[stage], phase, kStageWaitLimit)) failed = true;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const int lr = k + j * TEAMS + team;
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int c = v * TPR + t;
                    if (lr < rows && c < C) {
                        float2 d[NP], xh[NP];
                        values(s, oc, os, lr, c, rstd[j], d, xh);
#pragma unroll
                        for (int q = 0; q < NP; ++q) {
                            const float2 x = Pair<true>::mul(d[q], xh[q]);
                            dw[v][q] = Pair<true>::add(dw[v][q], x);
                            sum = Pair<true>::fma(x, f[v][q], sum);
                        }
                    }
                }
                part[j] = sum.x + sum.y;
            }
            constexpr int WIDTH = TPR < 32 ? TPR : 32;
#pragma unroll
            for (int o = WIDTH / 2; o > 0; o >>= 1)
#pragma unroll
                for (int j = 0; j < R; ++j) part[j] += __shfl_xor_sync(0xffffffffu, part[j], o);
            if constexpr (TPR > 32) {
                if ((t & 31) == 0)
#pragma unroll
                    for (int j = 0; j < R; ++j) red[flip][j][team][t >> 5] = part[j];
                sync_first<NT>();
#pragma unroll
                for (int j = 0; j < R; ++j) part[j] = sum_slots<W>(red[flip][j][team], t & 31);
            }
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const int lr = k + j * TEAMS + team;
                const float mc = part[j] * minus_inv;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int c = v * TPR + t;
                    if (lr < rows && c < C) {
                        float2 g[NP], xh[NP];
                        values(s, oc, os, lr, c, rstd[j], g, xh);
#pragma unroll
                        for (int q = 0; q < NP; ++q) {
                            g[q] = Pair<true>::fma(xh[q], make_float2(mc, mc), Pair<true>::mul(g[q], f[v][q]));
                            g[q] = Pair<true>::mul(g[q], make_float2(rstd[j], rstd[j]));
                        }
                        if constexpr (FUSED) {
                            float2 o[NP];
                            unpack<T>(lds128(s + lay.dres + ((size_t)lr * C + c) * 16), o);
#pragma unroll
                            for (int q = 0; q < NP; ++q) g[q] = Pair<true>::add(g[q], o[q]);
                        }
                        static_cast<uint4 *>(p.dx)[(r0 + lr) * C + c] = pack<T>(g);
                    }
                }
            }
        }
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[stage]);
        if (++stage == p.depth) stage = 0, phase ^= 1u;
    }
    if (failed) {  // no copy may land in shared memory that is another CTA's
        for (int i = max(0, mine - p.depth); i < mine; ++i) mbar_wait(&full[i % p.depth], (uint32_t)(i / p.depth) & 1u, kStageWaitLimit);
        if (p.status) *p.status = 1;
    }
    if (p.ws) {
        // the teams' sums of a column, one team after the other
        float *acc = reinterpret_cast<float *>(stages);
        for (int m = 0; m < TEAMS; ++m) {
            sync_first<NT>();
            if (team == m) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int c = v * TPR + t;
                    if (c < C) {
#pragma unroll
                        for (int q = 0; q < NP; ++q) {
                            float2 *a = reinterpret_cast<float2 *>(acc + c * E + 2 * q);
                            const float2 z = m == 0 ? dw[v][q] : Pair<true>::add(*a, dw[v][q]);
                            if (m == TEAMS - 1)
                                *reinterpret_cast<float2 *>(p.ws + (int64_t)blockIdx.x * p.N + c * E + 2 * q) = z;
                            else
                                *a = z;
                        }
                    }
                }
            }
        }
    }
}

// Rows of any alignment, value by value: persistent teams of TPR threads, a
// row at a time, K values a thread and their columns' sums in registers.
template <typename T, int TPR, int K, bool FUSED>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256) rows_bwd_lanes(const RowsBwdParams p) {
    constexpr int TEAMS = TPR >= 256 ? 1 : 256 / TPR, W = TPR / 32;
    __shared__ float red[2][TEAMS][W];
    extern __shared__ __align__(16) uint8_t stages[];  // several teams: [N] floats
    pdl_wait();
    pdl_trigger();
    const int team = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const int nb = (p.N + kBlock8 - 1) / kBlock8;
    float f[K], dw[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int j = k * TPR + t;
        f[k] = !p.w ? 1.f : j >= p.N ? 0.f : p.offset + (p.w32 ? load_w(static_cast<const float *>(p.w), j) : load_w(static_cast<const T *>(p.w), j));
        dw[k] = 0.f;
    }
    int flip = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * TEAMS; r0 < p.M; r0 += (int64_t)gridDim.x * TEAMS, flip ^= 1) {
        const int64_t row = r0 + team;
        const bool ok = row < p.M;
        const T *dy = static_cast<const T *>(p.dy) + row * p.N;
        const float rstd = ok ? p.rstd[row] : 0.f;
        // (all loads before the first use)
        T raw[K];
        int8_t code[K];
        uint8_t scale[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int j = k * TPR + t;
            if (ok && j < p.N) {
                raw[k] = dy[j];
                code[k] = (int8_t)p.codes[row * p.N + j];
                scale[k] = p.scales[row * nb + j / kBlock8];
            }
        }
        float d[K], xh[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const bool in = ok && k * TPR + t < p.N;
            d[k] = in ? load_elem(&raw[k], 0) : 0.f;
            xh[k] = in ? decode8(code[k]) * (rstd * from_codes8(scale[k])) : 0.f;
        }
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float x = d[k] * xh[k];
            dw[k] += x;
            s = fmaf(x, f[k], s);
        }
        const float c1 = team_allreduce<TPR>(s, red[flip][team], t) / (float)p.N;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int j = k * TPR + t;
            if (ok && j < p.N) {
                float v = rstd * fmaf(xh[k], -c1, d[k] * f[k]);
                if constexpr (FUSED) v += load_elem(static_cast<const T *>(p.dres) + row * p.N, j);
                store_elem(static_cast<T *>(p.dx) + row * p.N, j, v);
            }
        }
    }
    if (p.ws) {
        float *acc = reinterpret_cast<float *>(stages);
        for (int m = 0; m < TEAMS; ++m) {
            __syncthreads();
            if (team == m) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int j = k * TPR + t;
                    if (j < p.N) {
                        const float z = m == 0 ? dw[k] : acc[j] + dw[k];
                        if (m == TEAMS - 1)
                            p.ws[(int64_t)blockIdx.x * p.N + j] = z;
                        else
                            acc[j] = z;
                    }
                }
            }
        }
    }
}

// Any length: a CTA a row for dx, read twice ...
template <typename T, bool FUSED>
__global__ void __launch_bounds__(256) rows_bwd_any(const RowsBwdParams p) {
    __shared__ float red[32];
    pdl_wait();
    pdl_trigger();
    const int64_t row = blockIdx.x;
    const int nb = (p.N + kBlock8 - 1) / kBlock8;
    const T *dy = static_cast<const T *>(p.dy) + row * p.N;
    const float rstd = p.rstd[row];
    auto xhat = [&](int j) { return decode8((int8_t)p.codes[row * p.N + j]) * (rstd * from_codes8(p.scales[row * nb + j / kBlock8])); };
    auto weight = [&](int j) {
        return !p.w ? 1.f : p.offset + (p.w32 ? load_w(static_cast<const float *>(p.w), j) : load_w(static_cast<const T *>(p.w), j));
    };
    float s = 0.f;
    for (int j = threadIdx.x; j < p.N; j += 256) s = fmaf(load_elem(dy, j) * xhat(j), weight(j), s);
    const float c1 = cta_allreduce(s, red) / (float)p.N;
    for (int j = threadIdx.x; j < p.N; j += 256) {
        float v = rstd * fmaf(xhat(j), -c1, load_elem(dy, j) * weight(j));
        if constexpr (FUSED) v += load_elem(static_cast<const T *>(p.dres), row * p.N + j);
        store_elem(static_cast<T *>(p.dx), row * p.N + j, v);
    }
}

// ... and a thread a column over a chunk of rows for dw's partial rows. (It
// runs before rows_bwd_any: dx may be dy.)
template <typename T> __global__ void __launch_bounds__(256) rows_dw_any(const RowsBwdParams p, int rows) {
    pdl_wait();
    pdl_trigger();
    const int j = blockIdx.x * 256 + threadIdx.x;
    const int64_t r0 = (int64_t)blockIdx.y * rows, r1 = min(r0 + rows, (int64_t)p.M);
    const int nb = (p.N + kBlock8 - 1) / kBlock8;
    if (j < p.N) {
        float s = 0.f;
#pragma unroll 4
        for (int64_t r = r0; r < r1; ++r) {
            const float to = p.rstd[r] * from_codes8(p.scales[r * nb + j / kBlock8]);
            s = fmaf(load_elem(static_cast<const T *>(p.dy), r * p.N + j), decode8((int8_t)p.codes[r * p.N + j]) * to, s);
        }
        p.ws[(int64_t)blockIdx.y * p.N + j] = s;
    }
}

// ---------------------------------------------------------------- kernels --
// The teams that the kernels are compiled for: threads a row and chunks a
// thread, by the chunks they hold. A row takes the first that holds it.
#define ROWS_FWD_TEAMS(X) X(8, 1) X(32, 1) X(32, 2) X(64, 2) X(64, 4) X(128, 3) X(128, 4) X(256, 3) X(256, 4) X(512, 3) X(512, 4) X(1024, 4) X(1024, 8)
// (backward: and rows a team takes at once; 32 fp32 sums of dw a thread at most)
#define ROWS_BWD_TEAMS(X) \
    X(8, 1, 2) X(32, 1, 2) X(32, 2, 2) X(64, 2, 2) X(128, 2, 2) X(128, 3, 1) X(256, 2, 2) X(256, 3, 1) X(512, 2, 2) X(512, 3, 1) X(512, 4, 1)
#define ROWS_BWD_TEAMS4(X) X(512, 6, 1) X(512, 8, 1)

// Value by value: threads a row and values a thread.
#define ROWS_FWD_LANES(X) X(32, 1) X(32, 4) X(32, 16) X(128, 8) X(256, 8) X(256, 16) X(256, 32) X(512, 32)
// (backward of longer rows: a row's loads wait for one another's results in so few
// threads. 12000 x 5003: 600 us so, 420 in two launches of a CTA a row)
#define ROWS_BWD_LANES(X) X(32, 1) X(32, 4) X(32, 16) X(128, 8)

struct RowKernels {
    const void *fwd;
    int tpr, v, r;  // r 0: value by value; tpr 0: a CTA a row, any length
};

template <typename T, int SRC, bool KEEP> static RowKernels rows_fwd_pick(int N, bool wide) {
    const int C = N / Elem<T>::E;
    if (wide) {
#define X(tpr, v) \
    if (C <= tpr * v) return {(const void *)rows_fwd<T, tpr, v, SRC, KEEP>, tpr, v, 1};
        ROWS_FWD_TEAMS(X)
#undef X
    }
#define X(tpr, v) \
    if (N <= tpr * v) return {(const void *)rows_fwd_lanes<T, tpr, v, SRC, KEEP>, tpr, v, 0};
    ROWS_FWD_LANES(X)
#undef X
    return {(const void *)rows_fwd_any<T, SRC, KEEP>, 0, 0, 0};
}

template <typename T, bool FUSED> static RowKernels rows_bwd_pick(int N, bool wide) {
    const int C = N / Elem<T>::E;
    if (wide) {
#define X(tpr, v, r) \
    if (C <= tpr * v) return {(const void *)rows_bwd<T, tpr, v, r, FUSED>, tpr, v, r};
        ROWS_BWD_TEAMS(X)
        if constexpr (Elem<T>::E == 4) {
            ROWS_BWD_TEAMS4(X)
        }
#undef X
    }
#define X(tpr, v) \
    if (N <= tpr * v) return {(const void *)rows_bwd_lanes<T, tpr, v, FUSED>, tpr, v, 0};
    ROWS_BWD_LANES(X)
#undef X
    return {(const void *)rows_bwd_any<T, FUSED>, 0, 0, 0};
}

enum { kPackBlocks = 0, kPackAny, kUnpackBlocks, kUnpackAny, kEmbedRows, kDwAny };

template <typename T> static const void *rows_other_t(int which) {
    switch (which) {
    case kPackBlocks: return (const void *)pack_blocks<T>;
    case kPackAny: return (const void *)pack_any<T>;
    case kUnpackBlocks: return (const void *)unpack_blocks<T>;
    case kUnpackAny: return (const void *)unpack_any<T>;
    case kEmbedRows: return (const void *)embed_rows<T, 4>;
    default: return (const void *)rows_dw_any<T>;
    }
}
template <typename T> static RowKernels rows_fwd_t(int src, int N, bool wide) {
    return src == kSrcPlain ? rows_fwd_pick<T, kSrcPlain, true>(N, wide)
           : src == kSrcAdd ? rows_fwd_pick<T, kSrcAdd, true>(N, wide)
                            : rows_fwd_pick<T, kSrcEmbed, false>(N, wide);
}
template <typename T> static RowKernels rows_bwd_t(bool fused, int N, bool wide) {
    return fused ? rows_bwd_pick<T, true>(N, wide) : rows_bwd_pick<T, false>(N, wide);
}

#define ROWS_DECLARE(suf)                                   \
    const void *rows_other_##suf(int which);                \
    RowKernels rows_fwd_##suf(int src, int N, bool wide);   \
    RowKernels rows_bwd_##suf(bool fused, int N, bool wide);
ROWS_DECLARE(f32)
ROWS_DECLARE(bf16)
ROWS_DECLARE(f16)
#undef ROWS_DECLARE

}  // namespace rmsn
