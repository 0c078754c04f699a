// groupnorm_held.cuh -- group norm in one launch that reads its rows once: a
// cluster of CTAs holds what it normalises in shared memory.
//
// A cluster takes whole groups of one sample (all channels, or a span of them
// that begins on a 16-byte boundary) and each of its CTAs an equal share of
// the places, which comes into shared memory by asynchronous copies,
// kHeldStages pieces one behind the other: the sums begin with the first.
// Chunks are copied by the thread that later reads them, so no thread waits
// for another's; rows of any length and alignment are copied in bulk. (A bulk
// copy a row of a span instead took 31 us for 8 x 4096 x 320, the copies by
// chunks 19.) The CTAs' group sums meet in distributed shared memory, and the
// second pass reads shared memory.
//
// Bytes: x in, y out (forward), x and dy in, dx out: once each. 8 x 4096 x 320
// in bf16: 14.7 us forward (2.8 TB/s), 34 us the gradient with its finalizer
// (1.8 TB/s); load, sums and store follow one another in one round of CTAs.
#pragma once

#include "groupnorm_kernels.cuh"

namespace rmsn {

constexpr int kHeldThreads = 256;
constexpr int kHeldStages = 4;
constexpr int kHeldCtas = 16;                 // of a cluster at most
constexpr uint32_t kHeldWaitLimit = 1u << 20;  // polls of a piece's copies

struct HeldParams {
    GnParams g;      // rows: places a CTA takes
    int ctas;        // of a cluster
    int W, K, spans;  // channels and groups a cluster takes, clusters a sample
    uint32_t slab[2];  // bytes a CTA's share of x (or its codes) and of dy has in shared memory
    uint32_t scales;   // and of scale bytes
    int *status;
};

// A CTA's share of rows in shared memory. Chunks (E > 1): one behind the
// other, W / E a row. Single values: the 16-byte blocks that hold the share
// (rows of all channels are contiguous, from any address).
struct Slab {
    const char *src;
    uint8_t *dst;
    uint32_t off, row, piece, bytes;  // offset of the first row, bytes of a row, of a piece, of all
    __device__ __forceinline__ Slab(const void *base, int es, int64_t first_row, int C, int rows, uint8_t *to) {
        src = static_cast<const char *>(base) + first_row * C * es;
        dst = to;
        row = (uint32_t)C * es;
        const Cover c = cover16(src, (uint32_t)rows * row);
        src = c.src;
        off = c.off;
        bytes = rows > 0 ? c.bytes : 0u;
        piece = ((bytes + kHeldStages - 1) / kHeldStages + 15u) & ~15u;
    }
    __device__ __forceinline__ uint32_t piece_bytes(int i) const {
        const uint32_t at = (uint32_t)i * piece;
        return at < bytes ? min(piece, bytes - at) : 0u;
    }
    // rows that are there once pieces 0 .. i are
    __device__ __forceinline__ int ready(int i, int rows) const {
        const uint32_t end = (uint32_t)(i + 1) * piece;
        return end >= bytes ? rows : end > off ? min(rows, (int)((end - off) / row)) : 0;
    }
    __device__ __forceinline__ void fetch(int i, uint64_t *bar) const {
        const uint32_t at = (uint32_t)i * piece, n = piece_bytes(i);
        if (n > 0) bulk_g2s(dst + at, src + at, n, bar);
    }
};

// (16 bytes: past the L1)
template <int BYTES> __device__ __forceinline__ void copy_chunk(uint8_t *to, const void *from) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(to)), "l"(from), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until all but the latest `n` groups of this thread's copies have landed.
__device__ __forceinline__ void copies_wait(int n) {
    switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    }
}
static_assert(kHeldStages == 4, "copies_wait");

// Of a thread's n rows of a chunk column, those of pieces 0 .. i.
__device__ __forceinline__ int end_of(int n, int i) { return (n * (i + 1) + kHeldStages - 1) / kHeldStages; }

struct HeldPlace {
    int rank, b, c0, g0, rows;
    int64_t first;  // first row of the matrix
    __device__ __forceinline__ HeldPlace(const HeldParams &p) {
        const int unit = (int)blockIdx.x / p.ctas;
        rank = (int)blockIdx.x - unit * p.ctas;
        b = unit / p.spans;
        const int s = unit - b * p.spans;
        c0 = s * p.W;
        g0 = s * p.K;
        const int64_t r0 = (int64_t)rank * p.g.rows;
        rows = (int)max((int64_t)0, min((int64_t)p.g.rows, p.g.S - r0));
        first = (int64_t)b * p.g.S + r0;
    }
    static __device__ __forceinline__ int rows_of(const HeldParams &p, int r) {
        return (int)max((int64_t)0, min((int64_t)p.g.rows, p.g.S - (int64_t)r * p.g.rows));
    }
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <typename T, int E, int ACT, bool KEEP>
__global__ void __launch_bounds__(kHeldThreads, 2) gn_fwd_held(const HeldParams p) {
    extern __shared__ __align__(128) uint8_t held[];
    __shared__ __align__(8) uint64_t bar[kHeldStages];
    __shared__ bool failed;
    constexpr int CB = E * (int)sizeof(T);  // bytes of a chunk
    const GnParams &g = p.g;
    float *lane_mean = reinterpret_cast<float *>(held + p.slab[0]), *lane_m2 = lane_mean + kHeldThreads * E;
    float *ch_mean = lane_m2 + kHeldThreads * E, *ch_m2 = ch_mean + p.W;
    float2 *exch = reinterpret_cast<float2 *>(ch_m2 + p.W);
    float2 *stat = exch + p.ctas * p.K, *own = stat + p.K;
    const HeldPlace at(p);
    const Slab xs(g.x, sizeof(T), at.first, g.C, at.rows, held);
    if constexpr (E == 1) {
        if (threadIdx.x == 0) {
            failed = false;
            for (int i = 0; i < kHeldStages; ++i) mbar_init(&bar[i], 1);
            mbar_init_fence();
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncthreads();
    }
    cluster_arrive();  // by the exchange every CTA of the cluster has begun
    pdl_wait();
    pdl_trigger();
    const int CW = p.W / E;
    const Cut cut(CW, kHeldThreads);
    const uint32_t rows = smem_u32(held) + (E == 1 ? xs.off : 0u);
    const uint32_t pitch = (uint32_t)p.W * sizeof(T);
    if constexpr (E == 1) {
        if (threadIdx.x == 0)
            for (int i = 0; i < kHeldStages; ++i) {
                mbar_arrive_expect_tx(&bar[i], xs.piece_bytes(i));
                xs.fetch(i, &bar[i]);
            }
    }
    for (int t0 = 0; t0 < CW; t0 += cut.cols) {
        const int cc = t0 + cut.col;
        const bool in = cut.in && cc < CW;
        float K[E], s1[E], s2[E];
#pragma unroll
        for (int i = 0; i < E; ++i) K[i] = s1[i] = s2[i] = 0.f;
        const int n = in ? rows_of_lane(at.rows, cut.lane, cut.lanes) : 0;
        if constexpr (E > 1) {
            const T *x = static_cast<const T *>(g.x) + (at.first + cut.lane) * g.C + at.c0 + cc * E;
            uint8_t *to = held + (uint32_t)cut.lane * pitch + cc * CB;
            int k = 0;
            for (int i = 0; i < kHeldStages; ++i) {
                for (const int end = end_of(n, i); k < end; ++k)
                    copy_chunk<CB>(to + (uint32_t)(k * cut.lanes) * pitch, x + (int64_t)k * cut.lanes * g.C);
                copies_commit();
            }
        }
        const uint32_t from = rows + (uint32_t)cut.lane * pitch + cc * CB, step = (uint32_t)cut.lanes * pitch;
        for (int i = 0, k = 0; i < kHeldStages; ++i) {
            int end;  // of this thread's rows
            if constexpr (E > 1) {
                copies_wait(kHeldStages - 1 - i);
                end = end_of(n, i);
            } else {
                if (!mbar_wait(&bar[i], 0, kHeldWaitLimit)) failed = true;
                end = in ? rows_of_lane(xs.ready(i, at.rows), cut.lane, cut.lanes) : 0;
            }
            sum_rows<T, E>(from + (uint32_t)k * step, end - k, step, k, K, s1, s2);
            k = max(k, end);
        }
        lane_stats(n, K, s1, s2, lane_mean + threadIdx.x * E, lane_m2 + threadIdx.x * E);
        __syncthreads();
        join_lanes<kHeldThreads>(lane_mean, lane_m2, cut.cols * E, cut.lanes, at.rows);
        __syncthreads();
        for (int c = threadIdx.x; c < cut.cols * E && t0 * E + c < p.W; c += kHeldThreads) {
            ch_mean[t0 * E + c] = lane_mean[c];
            ch_m2[t0 * E + c] = lane_m2[c];
        }
        __syncthreads();
    }
    // a group's channels (all of at.rows places); then to every CTA of the cluster
    cluster_wait();
    const float inv_cg = 1.f / (float)g.cg;
    sum_groups<kHeldThreads>(
        0, p.W, g.cg,
        [&](int lo, int c) {  // about the first channel's mean
            const float d = ch_mean[c] - ch_mean[lo];
            return make_float2(d, fmaf((float)at.rows * d, d, ch_m2[c]));
        },
        [&](int k, int lo, int, float2 m) {
            const float d = m.x * inv_cg;
            own[k] = make_float2(ch_mean[lo] + d, at_least_0(m.y - (float)at.rows * m.x * d));
        });
    __syncthreads();
    for (int i = threadIdx.x; i < p.K * p.ctas; i += kHeldThreads) st_cluster2(&exch[at.rank * p.K + i % p.K], (uint32_t)(i / p.K), own[i % p.K]);
    cluster_sync();
    for (int k = threadIdx.x; k < p.K; k += kHeldThreads) {
        const float n = (float)g.S * (float)g.cg, ref = exch[k].x;
        float s = 0.f, m2 = 0.f;
        for (int r = 1; r < p.ctas; ++r) {
            const float cnt = (float)HeldPlace::rows_of(p, r);
            if (cnt > 0.f) s += cnt * (exch[r * p.K + k].x - ref);
        }
        const float m = ref + s / (float)g.S;
        for (int r = 0; r < p.ctas; ++r) {
            const float cnt = (float)HeldPlace::rows_of(p, r) * (float)g.cg;
            if (cnt > 0.f) {
                const float2 e = exch[r * p.K + k];
                const float d = e.x - m;
                m2 += fmaf(cnt * d, d, e.y);
            }
        }
        const float rs = 1.f / sqrtf(m2 / n + g.eps);
        stat[k] = make_float2(-m, rs);
        if (at.rank == 0) {
            g.mean[(int64_t)at.b * g.G + at.g0 + k] = m;
            g.rstd[(int64_t)at.b * g.G + at.g0 + k] = rs;
        }
    }
    __syncthreads();
    T *y = static_cast<T *>(g.out) + at.first * g.C + at.c0;
    for (int t0 = 0; t0 < CW; t0 += cut.cols) {
        const int cc = t0 + cut.col;
        if (!cut.in || cc >= CW) continue;
        float minus_mean[E], f[E], beta[E], gamma[E];
        groups_v(stat, cc * E, g.cg, g.magic, minus_mean, f);
        params_v<T>(g.gamma, g.w32, at.c0 + cc * E, 1.f, gamma);
        params_v<T>(g.beta, g.w32, at.c0 + cc * E, 0.f, beta);
        mul_v(f, gamma, f);
        uint32_t from = rows + (uint32_t)cut.lane * pitch + cc * CB;
        const uint32_t step = (uint32_t)cut.lanes * pitch;
        const int64_t out_step = (int64_t)cut.lanes * g.C;
        T *out = y + (int64_t)cut.lane * g.C + cc * E;
        int64_t row = at.first + cut.lane;
#pragma unroll 2
        for (int n = rows_of_lane(at.rows, cut.lane, cut.lanes); n > 0; --n, from += step, out += out_step, row += cut.lanes) {
            float v[E], z[E];
            const Vals<T, E> raw = held_chunk<T, E>(from);
            raw.get(v);
            gn_value<T, ACT>(v, minus_mean, f, beta, z);
            Vals<T, E> o;
            o.set(z);
            o.store(out);
            if constexpr (KEEP) {
                const int c = at.c0 + cc * E;
                keep_chunk<T, E>(raw.u, true, block_lanes<E>(), g.codes + row * g.C + c, g.scales + row * (g.C / kBlock8) + c / kBlock8);
            }
        }
    }
    if (E == 1 && failed && threadIdx.x == 0) {
        for (int i = 0; i < kHeldStages; ++i) mbar_wait(&bar[i], 0, kHeldWaitLimit);
        if (p.status) *p.status = 1;
    }
}

template <typename T, int E, int ACT, bool KEPT>
__global__ void __launch_bounds__(kHeldThreads, 2) gn_bwd_held(const HeldParams p) {
    extern __shared__ __align__(128) uint8_t held[];
    __shared__ __align__(8) uint64_t bar[kHeldStages];
    __shared__ bool failed;
    constexpr int CB = E * (int)sizeof(T);  // bytes of a chunk
    const GnParams &g = p.g;
    uint8_t *sc = held + p.slab[0] + p.slab[1];  // scale bytes [rows, nsc]
    float *lane_a = reinterpret_cast<float *>(sc + p.scales), *lane_s = lane_a + kHeldThreads * E;
    float *ch_a = lane_s + kHeldThreads * E, *ch_s = ch_a + p.W;
    float2 *exch = reinterpret_cast<float2 *>(ch_s + p.W);
    float2 *means = exch + p.ctas * p.K, *stat = means + p.K;
    const HeldPlace at(p);
    constexpr int XE = KEPT ? 1 : (int)sizeof(T);  // bytes of a value of x
    const Slab xs(KEPT ? (const void *)g.codes_in : g.x, XE, at.first, g.C, at.rows, held);
    const Slab ds(g.dy, sizeof(T), at.first, g.C, at.rows, held + p.slab[0]);
    if constexpr (E == 1) {
        if (threadIdx.x == 0) {
            failed = false;
            for (int i = 0; i < kHeldStages; ++i) mbar_init(&bar[i], 1);
            mbar_init_fence();
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncthreads();
    }
    cluster_arrive();
    pdl_wait();
    pdl_trigger();
    const int CW = p.W / E;
    const Cut cut(CW, kHeldThreads);
    const uint32_t xrows = smem_u32(held) + (E == 1 ? xs.off : 0u), drows = smem_u32(held) + p.slab[0] + (E == 1 ? ds.off : 0u),
                   srows = smem_u32(held) + p.slab[0] + p.slab[1];
    const uint32_t xpitch = (uint32_t)p.W * XE, dpitch = (uint32_t)p.W * sizeof(T);
    auto copy_column = [&](int cc, int n) {  // a chunk column's rows of this lane
        const int64_t first = (at.first + cut.lane) * g.C + at.c0 + cc * E;
        const char *x = (KEPT ? (const char *)g.codes_in : static_cast<const char *>(g.x)) + first * XE;
        const T *d = static_cast<const T *>(g.dy) + first;
        uint8_t *xto = held + (uint32_t)cut.lane * xpitch + cc * (E * XE), *dto = held + p.slab[0] + (uint32_t)cut.lane * dpitch + cc * CB;
        const int64_t step = (int64_t)cut.lanes * g.C;
        int k = 0;
        for (int i = 0; i < kHeldStages; ++i) {
            for (const int end = end_of(n, i); k < end; ++k) {
                copy_chunk<E * XE>(xto + (uint32_t)(k * cut.lanes) * xpitch, x + k * step * XE);
                copy_chunk<CB>(dto + (uint32_t)(k * cut.lanes) * dpitch, d + k * step);
            }
            copies_commit();
        }
    };
    if constexpr (E == 1) {
        if (threadIdx.x == 0)
            for (int i = 0; i < kHeldStages; ++i) {
                mbar_arrive_expect_tx(&bar[i], xs.piece_bytes(i) + ds.piece_bytes(i));
                xs.fetch(i, &bar[i]);
                ds.fetch(i, &bar[i]);
            }
    } else {
        copy_column(cut.col, cut.in ? rows_of_lane(at.rows, cut.lane, cut.lanes) : 0);
    }
    const int sc0 = at.c0 / kBlock8, nsc = KEPT ? (at.c0 + p.W - 1) / kBlock8 - sc0 + 1 : 0;
    if constexpr (KEPT) {
        const int all = (g.C + kBlock8 - 1) / kBlock8;
        for (int i = threadIdx.x; i < at.rows * nsc; i += kHeldThreads) {
            const int r = i / nsc;
            sc[i] = g.scales_in[(at.first + r) * all + sc0 + (i - r * nsc)];
        }
    }
    for (int k = threadIdx.x; k < p.K; k += kHeldThreads) {
        const int64_t i = (int64_t)at.b * g.G + at.g0 + k;
        stat[k] = make_float2(-g.mean[i], g.rstd[i]);
    }
    __syncthreads();
    // A chunk column's places in shared memory, from row to row.
    struct Walk {
        uint32_t x, d, s;
    };
    auto walk = [&](int r, int cc) {
        return Walk{xrows + (uint32_t)r * xpitch + cc * (E * XE), drows + (uint32_t)r * dpitch + cc * CB,
                    srows + (uint32_t)(r * nsc + (at.c0 + cc * E) / kBlock8 - sc0)};
    };
    const Walk step{(uint32_t)cut.lanes * xpitch, (uint32_t)cut.lanes * dpitch, (uint32_t)(cut.lanes * nsc)};
    // xhat and u of a chunk: what both passes form anew
    auto chunk = [&](Walk &w, const float (&minus_mean)[E], const float (&rstd)[E], const float (&gamma)[E], const float (&beta)[E],
                     float (&xhat)[E], float (&u)[E]) {
        if constexpr (KEPT)
            held_codes<E>(w.x, held_byte(w.s), xhat);
        else
            held_values<T, E>(w.x, xhat);
        held_values<T, E>(w.d, u);
        w.x += step.x, w.d += step.d;
        if constexpr (KEPT) w.s += step.s;
        gn_slope<T, ACT>(xhat, u, minus_mean, rstd, gamma, beta);
    };
    auto constants = [&](int cc, float (&minus_mean)[E], float (&rstd)[E], float (&gamma)[E], float (&beta)[E]) {
        groups_v(stat, cc * E, g.cg, g.magic, minus_mean, rstd);
        params_v<T>(g.gamma, g.w32, at.c0 + cc * E, 1.f, gamma);
        params_v<T>(g.beta, g.w32, at.c0 + cc * E, 0.f, beta);
    };
    float *out = g.parts + ((int64_t)at.b * p.ctas + at.rank) * 2 * g.C;
    for (int t0 = 0; t0 < CW; t0 += cut.cols) {
        const int cc = t0 + cut.col;
        const bool in = cut.in && cc < CW;
        float a[E], s[E];
#pragma unroll
        for (int i = 0; i < E; ++i) a[i] = s[i] = 0.f;
        float minus_mean[E], rstd[E], gamma[E], beta[E];
        const int n = in ? rows_of_lane(at.rows, cut.lane, cut.lanes) : 0;
        if constexpr (E > 1) {
            if (t0 > 0) copy_column(cc, n);
        }
        if (in) constants(cc, minus_mean, rstd, gamma, beta);
        Walk w = walk(cut.lane, cc);
        for (int i = 0, k = 0; i < kHeldStages; ++i) {
            int end;  // of this thread's rows
            if constexpr (E > 1) {
                copies_wait(kHeldStages - 1 - i);
                end = end_of(n, i);
            } else {
                if (!mbar_wait(&bar[i], 0, kHeldWaitLimit)) failed = true;
                end = in ? rows_of_lane(min(xs.ready(i, at.rows), ds.ready(i, at.rows)), cut.lane, cut.lanes) : 0;
            }
#pragma unroll 2
            for (; k < end; ++k) {
                float xhat[E], u[E];
                chunk(w, minus_mean, rstd, gamma, beta, xhat, u);
                fma_v(u, xhat, a, a);
                add_v(s, u, s);
            }
        }
        put_v(lane_a + threadIdx.x * E, a);
        put_v(lane_s + threadIdx.x * E, s);
        __syncthreads();
        const int width = cut.cols * E;
        for (int c = threadIdx.x; c < width && t0 * E + c < p.W; c += kHeldThreads) {
            float ta = lane_a[c], ts = lane_s[c];
#pragma unroll 8
            for (int l = 1; l < cut.lanes; ++l) {
                ta += lane_a[l * width + c];
                ts += lane_s[l * width + c];
            }
            const int ch = t0 * E + c;
            if (g.parts) {
                out[at.c0 + ch] = ta;
                out[g.C + at.c0 + ch] = ts;
            }
            const float ga = param<T>(g.gamma, g.w32, at.c0 + ch, 1.f);
            ch_a[ch] = ta * ga;
            ch_s[ch] = ts * ga;
        }
        __syncthreads();
    }
    cluster_wait();
    sum_groups<kHeldThreads>(
        0, p.W, g.cg, [&](int, int c) { return make_float2(ch_s[c], ch_a[c]); }, [&](int k, int, int, float2 m) { means[k] = m; });
    __syncthreads();
    for (int i = threadIdx.x; i < p.K * p.ctas; i += kHeldThreads) st_cluster2(&exch[at.rank * p.K + i % p.K], (uint32_t)(i / p.K), means[i % p.K]);
    cluster_sync();
    for (int k = threadIdx.x; k < p.K; k += kHeldThreads) {
        const float n = (float)g.S * (float)g.cg;
        float2 m = exch[k];
        for (int r = 1; r < p.ctas; ++r) m = add2(m, exch[r * p.K + k]);
        means[k] = make_float2(-m.x / n, -m.y / n);
    }
    __syncthreads();
    T *dx = static_cast<T *>(g.out) + at.first * g.C + at.c0;
    for (int t0 = 0; t0 < CW; t0 += cut.cols) {
        const int cc = t0 + cut.col;
        if (!cut.in || cc >= CW) continue;
        float minus_mean[E], rstd[E], gamma[E], beta[E];
        constants(cc, minus_mean, rstd, gamma, beta);
        float m1[E], m2[E];
        groups_v(means, cc * E, g.cg, g.magic, m1, m2);
        Walk w = walk(cut.lane, cc);
        const int64_t out_step = (int64_t)cut.lanes * g.C;
        T *to = dx + (int64_t)cut.lane * g.C + cc * E;
#pragma unroll 1
        for (int n = rows_of_lane(at.rows, cut.lane, cut.lanes); n > 0; --n, to += out_step) {
            float xhat[E], u[E];
            chunk(w, minus_mean, rstd, gamma, beta, xhat, u);
            gn_dx(xhat, u, rstd, gamma, m1, m2);
            Vals<T, E> o;
            o.set(u);
            o.store(to);
        }
    }
    if (E == 1 && failed && threadIdx.x == 0) {
        for (int i = 0; i < kHeldStages; ++i) mbar_wait(&bar[i], 0, kHeldWaitLimit);
        if (p.status) *p.status = 1;
    }
}

// (keeping x in the same pass: whole 16-byte chunks only)
template <typename T, int E, int ACT> static const void *held_fwd() {
    if constexpr (E > 1)
        return (const void *)gn_fwd_held<T, E, ACT, true>;
    else
        return nullptr;
}
template <typename T, int E> static const void *gn_held_e(bool backward, int act, bool kept) {
#define HELD(A)                                                                                        \
    (backward ? (kept ? (const void *)gn_bwd_held<T, E, A, true> : (const void *)gn_bwd_held<T, E, A, false>) \
     : kept   ? held_fwd<T, E, A>()                                                                    \
              : (const void *)gn_fwd_held<T, E, A, false>)
    return act == kActSilu ? HELD(kActSilu) : act == kActGelu ? HELD(kActGelu) : HELD(kActNone);
#undef HELD
}
template <typename T> static const void *gn_held_t(bool backward, int chunk, int act, bool kept) {
    if constexpr (sizeof(T) == 2) {
        if (chunk == 8) return gn_held_e<T, 8>(backward, act, kept);
    }
    return chunk == 4 ? gn_held_e<T, 4>(backward, act, kept) : gn_held_e<T, 1>(backward, act, kept);
}

}  // namespace rmsn
