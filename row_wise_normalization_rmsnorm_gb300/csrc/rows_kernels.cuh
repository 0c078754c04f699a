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
// forward with its checkpoint (x, y, code), 5.03 for the backward.
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
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = v * TPR + t;
        const bool in = ok && c < C;
        float2 a[NP];
        unpack<T>(h[v], a);
        if constexpr (KEEP) {
            float f[E];
#pragma unroll
            for (int q = 0; q < NP; ++q) f[2 * q] = a[q].x, f[2 * q + 1] = a[q].y;
            const int64_t blocks = (p.N + kBlock8 - 1) / kBlock8;
            keep_chunk<T, E>(f, in, p.codes + row * p.N + (int64_t)c * E, p.scales + row * blocks + c * E / kBlock8);
        }
        if (in) {
            float2 f[NP];
            weights_at<T>(p.w, p.w32, c, p.offset, f);
#pragma unroll
            for (int q = 0; q < NP; ++q) a[q] = Pair<true>::mul(Pair<true>::mul(a[q], make_float2(rstd, rstd)), f[q]);
            static_cast<uint4 *>(p.y)[row * C + c] = pack<T>(a);
        }
    }
}

// Rows of any length and alignment: a CTA a row, value by value. Consecutive
// lanes take consecutive values, so a warp's 32 are a block.
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
            if (in) p.codes[row * p.N + j] = (uint8_t)code8(v, to_codes8(b));
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
    constexpr int E = Elem<T>::E, NP = Elem<T>::NP;
    pdl_wait();
    pdl_trigger();
    const int64_t c0 = (int64_t)blockIdx.x * 256 * kPackChunks + threadIdx.x;
    uint4 r[kPackChunks];
#pragma unroll
    for (int k = 0; k < kPackChunks; ++k) r[k] = c0 + 256 * k < chunks ? ld_stream(x + c0 + 256 * k) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < kPackChunks; ++k) {
        const int64_t c = c0 + 256 * k;
        float2 a[NP];
        float f[E];
        unpack<T>(r[k], a);
#pragma unroll
        for (int q = 0; q < NP; ++q) f[2 * q] = a[q].x, f[2 * q + 1] = a[q].y;
        keep_chunk<T, E>(f, c < chunks, codes + c * E, scales + c * E / kBlock8);
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

// Rows of any length and alignment: a warp a block at a time, lane by lane.
template <typename T>
__global__ void __launch_bounds__(256) pack_any(const T *x, uint8_t *codes, uint8_t *scales, int64_t M, int N) {
    pdl_wait();
    pdl_trigger();
    const int blocks = (N + kBlock8 - 1) / kBlock8, lane = threadIdx.x & 31;
    const int64_t first = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * kPackChunks;
    const int64_t all = M * blocks;
    float v[kPackChunks];
#pragma unroll
    for (int k = 0; k < kPackChunks; ++k) {
        const int64_t i = first + k, row = i / blocks;
        const int j = (int)(i - row * blocks) * kBlock8 + lane;
        v[k] = i < all && j < N ? load_elem(x, row * N + j) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kPackChunks; ++k) {
        const int64_t i = first + k, row = i / blocks;
        const int j = (int)(i - row * blocks) * kBlock8 + lane;
        const uint32_t b = scale8<T>(__reduce_max_sync(0xffffffffu, abs_bits(v[k])));
        if (i < all) {
            if (j < N) codes[row * N + j] = (uint8_t)code8(v[k], to_codes8(b));
            if (lane == 0) scales[i] = (uint8_t)b;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256) unpack_any(const uint8_t *codes, const uint8_t *scales, T *x, int64_t M, int N) {
    pdl_wait();
    pdl_trigger();
    const int blocks = (N + kBlock8 - 1) / kBlock8, lane = threadIdx.x & 31;
    const int64_t first = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * kPackChunks;
    const int64_t all = M * blocks;
#pragma unroll
    for (int k = 0; k < kPackChunks; ++k) {
        const int64_t i = first + k, row = i / blocks;
        const int j = (int)(i - row * blocks) * kBlock8 + lane;
        if (i < all && j < N) store_elem(x, row * N + j, decode8((int8_t)codes[row * N + j]) * from_codes8(scales[i]));
    }
}

// ---------------------------------------------------------------- backward --
// Persistent: CTA i takes blocks of `stage_rows` rows i, i + grid, ..., which
// bulk copies bring into shared memory `depth` blocks ahead; a team of TPR
// threads takes a row, holds its chunks in registers between the sum and dx,
// and keeps dw's sums of its columns until the end. Codes, scales and rstd of
// a block start anywhere: the 16-byte blocks that hold them are copied.
__host__ __device__ constexpr uint32_t up16(uint32_t n) { return (n + 15u) & ~15u; }

struct StageLayout {  // byte offsets in a stage
    uint32_t dres, codes, scales, rstd, bytes;
    __host__ __device__ StageLayout(int rows, int N, int es, bool fused) {
        const uint32_t row = (uint32_t)rows * N, blocks = (uint32_t)rows * ((N + kBlock8 - 1) / kBlock8);
        dres = row * es;
        codes = dres + (fused ? row * es : 0u);
        scales = codes + up16(row + 15u);
        rstd = scales + up16(blocks + 15u);
        bytes = rstd + up16(rows * 4u + 15u);
    }
};

constexpr uint32_t kStageWaitLimit = 1u << 20;  // polls of a stage's copies (each may suspend the thread for a while)

template <typename T, int TPR, int V, bool FUSED>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256, TPR > 256 ? 1 : 2) rows_bwd(const RowsBwdParams p) {
    constexpr int E = Elem<T>::E, NP = Elem<T>::NP, TEAMS = TPR >= 256 ? 1 : 256 / TPR, W = TPR > 32 ? TPR / 32 : 1;
    extern __shared__ __align__(128) uint8_t stages[];
    __shared__ float red[2][TEAMS][W];
    __shared__ __align__(8) uint64_t full[8];
    const int team = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const int C = p.N / E, nb = (p.N + kBlock8 - 1) / kBlock8;
    const StageLayout lay(p.stage_rows, p.N, sizeof(T), FUSED);
    const int blocks = (p.M + p.stage_rows - 1) / p.stage_rows;
    const int mine = blocks > (int)blockIdx.x ? (blocks - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.depth; ++i) mbar_init(&full[i], 1);
        mbar_init_fence();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    auto fetch = [&](int i) {  // this CTA's i-th block, by one thread
        uint8_t *s = stages + (size_t)(i % p.depth) * lay.bytes;
        uint64_t *bar = &full[i % p.depth];
        const int64_t r0 = ((int64_t)blockIdx.x + (int64_t)i * gridDim.x) * p.stage_rows;
        const uint32_t rows = (uint32_t)min((int64_t)p.stage_rows, p.M - r0);
        const uint32_t bytes = rows * (uint32_t)p.N * sizeof(T);
        const Cover cc = cover16(p.codes + r0 * p.N, rows * p.N), cs = cover16(p.scales + r0 * nb, rows * nb),
                    cr = cover16(p.rstd + r0, rows * 4u);
        mbar_arrive_expect_tx(bar, bytes * (FUSED ? 2 : 1) + cc.bytes + cs.bytes + cr.bytes);
        bulk_g2s(s, static_cast<const T *>(p.dy) + r0 * p.N, bytes, bar);
        if (FUSED) bulk_g2s(s + lay.dres, static_cast<const T *>(p.dres) + r0 * p.N, bytes, bar);
        bulk_g2s(s + lay.codes, cc.src, cc.bytes, bar);
        bulk_g2s(s + lay.scales, cs.src, cs.bytes, bar);
        bulk_g2s(s + lay.rstd, cr.src, cr.bytes, bar);
    };
    if (threadIdx.x == 0)
        for (int i = 0; i < p.depth && i < mine; ++i) fetch(i);
    float2 f[V][NP], dw[V][NP];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = v * TPR + t;
#pragma unroll
        for (int q = 0; q < NP; ++q) f[v][q] = dw[v][q] = make_float2(0.f, 0.f);
        if (c < C) weights_at<T>(p.w, p.w32, c, p.offset, f[v]);
    }
    int flip = 0;
    bool failed = false;
    for (int i = 0; i < mine; ++i) {
        const uint8_t *s = stages + (size_t)(i % p.depth) * lay.bytes;
        if (!failed && !mbar_wait(&full[i % p.depth], (uint32_t)(i / p.depth) & 1u, kStageWaitLimit)) failed = true;
        const int64_t r0 = ((int64_t)blockIdx.x + (int64_t)i * gridDim.x) * p.stage_rows;
        const uint32_t oc = addr_mod16(p.codes + r0 * p.N), os = addr_mod16(p.scales + r0 * nb), orr = addr_mod16(p.rstd + r0);
        for (int k = 0; k < p.stage_rows; k += TEAMS, flip ^= 1) {
            const int lr = k + team;
            const bool ok = lr < p.stage_rows && r0 + lr < p.M;
            uint4 d[V], dr[FUSED ? V : 1];
            float2 xh[V][NP];
            float rstd = 0.f;
            float2 sum = make_float2(0.f, 0.f);
            if (ok) rstd = *reinterpret_cast<const float *>(s + lay.rstd + orr + lr * 4);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = v * TPR + t;
                if (ok && c < C) {
                    const uint32_t at = (uint32_t)lr * C + c;
                    d[v] = lds128(s + (size_t)at * 16);
                    if constexpr (FUSED) dr[v] = lds128(s + lay.dres + (size_t)at * 16);
                    const uint8_t *code = s + lay.codes + oc + at * E;
                    const float to = rstd * from_codes8(s[lay.scales + os + lr * nb + c * E / kBlock8]);
                    float x[E];
#pragma unroll
                    for (int e = 0; e < E / 4; ++e) {
                        float q4[4];
                        decode8x4(*reinterpret_cast<const uint32_t *>(code + 4 * e), q4);
#pragma unroll
                        for (int m = 0; m < 4; ++m) x[4 * e + m] = q4[m];
                    }
                    float2 dyv[NP];
                    unpack<T>(d[v], dyv);
#pragma unroll
                    for (int q = 0; q < NP; ++q) {
                        xh[v][q] = Pair<true>::mul(make_float2(x[2 * q], x[2 * q + 1]), make_float2(to, to));
                        const float2 dx = Pair<true>::mul(dyv[q], xh[v][q]);
                        dw[v][q] = Pair<true>::add(dw[v][q], dx);
                        sum = Pair<true>::fma(dx, f[v][q], sum);
                    }
                }
            }
            const float c1 = team_allreduce<TPR>(sum.x + sum.y, red[flip][team], t) / (float)p.N;
            if (k + TEAMS >= p.stage_rows) {
                // every thread holds its part of the last rows: the stage is free
                if constexpr (TPR <= 32) __syncthreads();
                if (threadIdx.x == 0 && i + p.depth < mine && !failed) {
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    fetch(i + p.depth);
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = v * TPR + t;
                if (ok && c < C) {
                    float2 g[NP], o[NP];
                    unpack<T>(d[v], g);
                    if constexpr (FUSED) unpack<T>(dr[v], o);
#pragma unroll
                    for (int q = 0; q < NP; ++q) {
                        const float2 gw = Pair<true>::mul(g[q], f[v][q]);
                        const float2 e = Pair<true>::fma(xh[v][q], make_float2(-c1, -c1), gw);
                        g[q] = FUSED ? Pair<true>::fma(e, make_float2(rstd, rstd), o[q]) : Pair<true>::mul(e, make_float2(rstd, rstd));
                    }
                    static_cast<uint4 *>(p.dx)[(r0 + lr) * C + c] = pack<T>(g);
                }
            }
        }
    }
    if (failed) {  // no copy may land in shared memory that is another CTA's
        for (int i = 0; i < p.depth && i < mine; ++i) mbar_wait(&full[i], (uint32_t)((mine - 1 - i) / p.depth) & 1u, kStageWaitLimit);
        if (p.status) *p.status = 1;
    }
    if (p.ws) {
        // the teams' sums of a column, one team after the other
        float *acc = reinterpret_cast<float *>(stages);
        for (int m = 0; m < TEAMS; ++m) {
            __syncthreads();
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

// Any length and alignment: a CTA a row for dx ...
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
struct TeamSize {
    int tpr, v;
};
#define ROWS_FWD_TEAMS(X) X(8, 1) X(32, 1) X(32, 2) X(64, 2) X(64, 4) X(128, 3) X(128, 4) X(256, 3) X(256, 4) X(512, 3) X(512, 4) X(1024, 4) X(1024, 8)
// (32 fp32 sums of dw a thread at most: 4 chunks of 8 values, 8 of 4)
#define ROWS_BWD_TEAMS(X) X(8, 1) X(32, 1) X(32, 2) X(64, 2) X(64, 4) X(128, 3) X(128, 4) X(256, 3) X(256, 4) X(512, 3) X(512, 4)
#define ROWS_BWD_TEAMS4(X) X(512, 6) X(512, 8)

struct RowKernels {
    const void *fwd;
    int tpr, v;  // 0: a CTA a row, any length
};

template <typename T, int SRC, bool KEEP> static RowKernels rows_fwd_pick(int C, bool wide) {
    if (wide) {
#define X(tpr, v) \
    if (C <= tpr * v) return {(const void *)rows_fwd<T, tpr, v, SRC, KEEP>, tpr, v};
        ROWS_FWD_TEAMS(X)
#undef X
    }
    return {(const void *)rows_fwd_any<T, SRC, KEEP>, 0, 0};
}

template <typename T, bool FUSED> static RowKernels rows_bwd_pick(int C, bool wide) {
    if (wide) {
#define X(tpr, v) \
    if (C <= tpr * v) return {(const void *)rows_bwd<T, tpr, v, FUSED>, tpr, v};
        ROWS_BWD_TEAMS(X)
        if constexpr (Elem<T>::E == 4) {
            ROWS_BWD_TEAMS4(X)
        }
#undef X
    }
    return {(const void *)rows_bwd_any<T, FUSED>, 0, 0};
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
template <typename T> static RowKernels rows_fwd_t(int src, int C, bool wide) {
    return src == kSrcPlain ? rows_fwd_pick<T, kSrcPlain, true>(C, wide)
           : src == kSrcAdd ? rows_fwd_pick<T, kSrcAdd, true>(C, wide)
                            : rows_fwd_pick<T, kSrcEmbed, false>(C, wide);
}
template <typename T> static RowKernels rows_bwd_t(bool fused, int C, bool wide) {
    return fused ? rows_bwd_pick<T, true>(C, wide) : rows_bwd_pick<T, false>(C, wide);
}

#define ROWS_DECLARE(suf)                                   \
    const void *rows_other_##suf(int which);                \
    RowKernels rows_fwd_##suf(int src, int C, bool wide);   \
    RowKernels rows_bwd_##suf(bool fused, int C, bool wide);
ROWS_DECLARE(f32)
ROWS_DECLARE(bf16)
ROWS_DECLARE(f16)
#undef ROWS_DECLARE

}  // namespace rmsn
