// groupnorm_kernels.cuh -- group norm over rows with the channels last, with
// an activation behind it: forward and backward.
//
//   x [B, S, C], group g of a sample: its S places' channels g C/G .. (g+1) C/G
//   mean, var  over the group's n = S C/G values,  rstd = 1 / sqrt(var + eps)
//   xhat = (x - mean) rstd,   z = xhat gamma + beta,   y = act(z)
//   backward: u = dy act'(z),  dgamma_c = sum u xhat,  dbeta_c = sum u  (over b, s)
//             dx = rstd (u gamma - (1/n) sum_group u gamma - xhat (1/n) sum_group u gamma xhat)
//
// Channels lie next to one another and groups are narrow (10 channels of bf16
// are 20 bytes), so a CTA takes whole rows, and a thread keeps to one chunk of
// neighbouring channels while it walks down its share of the rows: loads are
// contiguous over the CTA whatever the groups are, and a channel's constants
// stay in registers. Sums are taken a channel apart and meet in groups only at
// the end, so a group may begin inside a chunk.
#pragma once

#include "rows8.cuh"

namespace rmsn {

enum { kActNone = 0, kActSilu = 1, kActGelu = 2 };

struct GnParams {
    const void *x, *dy;
    const uint8_t *codes_in;   // x in 8 bits, in the place of x
    const uint8_t *scales_in;
    const void *gamma, *beta;  // NULL: 1 and 0
    void *out;                 // y or dx
    float *mean, *rstd;        // [B, G]
    uint8_t *codes, *scales;   // x kept in 8 bits (forward) or NULL
    float *parts;              // backward: [pieces, 2, C], a piece's channel sums of u xhat and of u (NULL: not wanted)
    int64_t S;
    int B, C, G, cg;           // cg = C / G
    int rows;                  // places a CTA takes
    int w32;
    uint32_t magic;            // ceil(2^32 / cg), 0 where cg is 1
    float eps;
};

// ------------------------------------------------------------ E-wide access --

template <int BYTES> struct Word;
template <> struct Word<16> { using type = uint4; };
template <> struct Word<8> { using type = uint2; };
template <> struct Word<4> { using type = uint32_t; };
template <> struct Word<2> { using type = uint16_t; };

template <typename T> __device__ __forceinline__ float widen(T v);
template <> __device__ __forceinline__ float widen<float>(float v) { return v; }
template <> __device__ __forceinline__ float widen<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// E values that lie together, as one access.
template <typename T, int E> struct Vals {
    using W = typename Word<E * (int)sizeof(T)>::type;
    W w;
    __device__ __forceinline__ void load(const T *p) { w = *reinterpret_cast<const W *>(p); }
    __device__ __forceinline__ void load_last(const T *p) { w = __ldcs(reinterpret_cast<const W *>(p)); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<W *>(p) = w; }
    __device__ __forceinline__ void get(float (&v)[E]) const {
        if constexpr (E == Elem<T>::E) {
            float2 q[Elem<T>::NP];
            unpack<T>(w, q);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) v[2 * i] = q[i].x, v[2 * i + 1] = q[i].y;
        } else {
            const T *t = reinterpret_cast<const T *>(&w);
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = widen<T>(t[i]);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[E]) {
        if constexpr (E == Elem<T>::E) {
            float2 q[Elem<T>::NP];
#pragma unroll
            for (int i = 0; i < E / 2; ++i) q[i] = make_float2(v[2 * i], v[2 * i + 1]);
            w = pack<T>(q);
        } else {
            T *t = reinterpret_cast<T *>(&w);
#pragma unroll
            for (int i = 0; i < E; ++i) store_elem(t, i, v[i]);
        }
    }
};

// E kept values: their codes and their block's scale.
template <int E> struct Kept {
    using W = typename std::conditional<E == 8, uint2, typename std::conditional<E == 4, uint32_t, uint8_t>::type>::type;
    W w;
    uint32_t b;
    __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *scales, int64_t row, int C, int c) {
        w = *reinterpret_cast<const W *>(codes + row * C + c);
        b = scales[row * ((C + kBlock8 - 1) / kBlock8) + c / kBlock8];
    }
    __device__ __forceinline__ void get(float (&v)[E]) const {
        const float f = from_codes8(b);
        if constexpr (E == 8) {
            float lo[4], hi[4];
            decode8x4(w.x, lo);
            decode8x4(w.y, hi);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = lo[i] * f, v[4 + i] = hi[i] * f;
        } else if constexpr (E == 4) {
            decode8x4(w, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] *= f;
        } else {
            v[0] = decode8((int8_t)w) * f;
        }
    }
};

template <typename T> __device__ __forceinline__ float param(const void *w, int w32, int c, float none) {
    if (!w) return none;
    return w32 ? static_cast<const float *>(w)[c] : widen<T>(static_cast<const T *>(w)[c]);
}

// ---------------------------------------------------------- chunk arithmetic --
// E values at once, in pairs where there are two (f32x2 instructions: these
// kernels are as near to their instruction rate as to memory's).
template <int E> __device__ __forceinline__ void fma_v(const float (&a)[E], const float (&b)[E], const float (&c)[E], float (&d)[E]) {
    if constexpr (E == 1) {
        d[0] = fmaf(a[0], b[0], c[0]);
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const float2 r = Pair<true>::fma(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]), make_float2(c[i], c[i + 1]));
            d[i] = r.x, d[i + 1] = r.y;
        }
    }
}
template <int E> __device__ __forceinline__ void mul_v(const float (&a)[E], const float (&b)[E], float (&d)[E]) {
    if constexpr (E == 1) {
        d[0] = a[0] * b[0];
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const float2 r = Pair<true>::mul(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
            d[i] = r.x, d[i + 1] = r.y;
        }
    }
}
template <int E> __device__ __forceinline__ void add_v(const float (&a)[E], const float (&b)[E], float (&d)[E]) {
    if constexpr (E == 1) {
        d[0] = a[0] + b[0];
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const float2 r = Pair<true>::add(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
            d[i] = r.x, d[i + 1] = r.y;
        }
    }
}
template <int E> __device__ __forceinline__ void fill_v(float v, float (&d)[E]) {
#pragma unroll
    for (int i = 0; i < E; ++i) d[i] = v;
}

// ------------------------------------------------------------- activations --
__device__ __forceinline__ float exp2_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// The sigmoids of E values. For 16-bit rows one reciprocal serves two
// (1 / a = b / (a b)): the special-function unit, 16 results a clock and SM,
// bounds these kernels next to memory, and so it gives 1.5 results a value
// instead of 2. z is held at -43, where the sigmoid is 2^-62 and a b still
// finite. (fmaxf drops a NaN; z, which every result is multiplied by, brings
// it back.) fp32 rows take the accurate exponential.
template <typename T, int E> __device__ __forceinline__ void sigmoid_v(const float (&z)[E], float (&p)[E]) {
    if constexpr (std::is_same<T, float>::value) {
#pragma unroll
        for (int i = 0; i < E; ++i) p[i] = rcp_fast(1.f + expf(-z[i]));
    } else if constexpr (E == 1) {
        p[0] = rcp_fast(1.f + exp2_fast(-1.4426950f * fmaxf(z[0], -43.f)));
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) p[i] = fmaxf(z[i], -43.f);
        float k[E], one[E];
        fill_v(-1.4426950f, k);
        fill_v(1.f, one);
        mul_v(p, k, p);
#pragma unroll
        for (int i = 0; i < E; ++i) p[i] = exp2_fast(p[i]);
        add_v(p, one, p);
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const float r = rcp_fast(p[i] * p[i + 1]);
            const float2 q = Pair<true>::mul(make_float2(r, r), make_float2(p[i + 1], p[i]));
            p[i] = q.x, p[i + 1] = q.y;
        }
    }
}
__device__ __forceinline__ float gelu_of(float z) { return 0.5f * z * (1.f + erff(z * 0.70710678f)); }
__device__ __forceinline__ float gelu_slope(float z) {
    return 0.5f * (1.f + erff(z * 0.70710678f)) + z * __expf(-0.5f * z * z) * 0.39894228f;
}

// act(z), act'(z) in place.
template <typename T, int ACT, int E> __device__ __forceinline__ void act_of(float (&z)[E]) {
    if constexpr (ACT == kActSilu) {
        float p[E];
        sigmoid_v<T>(z, p);
        mul_v(z, p, z);
    } else if constexpr (ACT == kActGelu) {
#pragma unroll
        for (int i = 0; i < E; ++i) z[i] = gelu_of(z[i]);
    }
}
template <typename T, int ACT, int E> __device__ __forceinline__ void act_slope(float (&z)[E]) {
    if constexpr (ACT == kActSilu) {  // p (1 + z (1 - p))
        float p[E], one[E], minus[E], q[E];
        sigmoid_v<T>(z, p);
        fill_v(1.f, one);
        fill_v(-1.f, minus);
        fma_v(p, minus, one, q);
        fma_v(z, q, one, q);
        mul_v(p, q, z);
    } else if constexpr (ACT == kActGelu) {
#pragma unroll
        for (int i = 0; i < E; ++i) z[i] = gelu_slope(z[i]);
    } else {
        fill_v(1.f, z);
    }
}

// gamma and beta of E channels from c0 (NULL: 1 and 0).
template <typename T, int E> __device__ __forceinline__ void params_v(const void *w, int w32, int c0, float none, float (&v)[E]) {
    if (!w) {
        fill_v(none, v);
    } else if (w32) {
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = static_cast<const float *>(w)[c0 + i];
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = widen<T>(static_cast<const T *>(w)[c0 + i]);
    }
}
// A group's pair of values for each of E channels from c0 (of the groups at
// `of`): one look where the chunk lies in a group.
template <int E> __device__ __forceinline__ void groups_v(const float2 *of, int c0, int cg, uint32_t magic, float (&x)[E], float (&y)[E]) {
    // c / cg for c < 2^16 (magic = ceil(2^32 / cg), 0 where cg is 1)
    auto group = [&](int c) { return magic ? (int)__umulhi((uint32_t)c, magic) : c; };
    if (cg % E == 0) {
        const float2 s = of[group(c0)];
        fill_v(s.x, x);
        fill_v(s.y, y);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float2 s = of[group(c0 + i)];
            x[i] = s.x;
            y[i] = s.y;
        }
    }
}

// y = act((v - mean) f + beta), f = rstd gamma; v and the result in z.
template <typename T, int ACT, int E>
__device__ __forceinline__ void gn_value(const float (&v)[E], const float (&minus_mean)[E], const float (&f)[E], const float (&beta)[E], float (&z)[E]) {
    add_v(v, minus_mean, z);
    fma_v(z, f, beta, z);
    act_of<T, ACT>(z);
}
// v becomes xhat and g (dy) u = dy act'(xhat gamma + beta).
template <typename T, int ACT, int E>
__device__ __forceinline__ void gn_slope(float (&v)[E], float (&g)[E], const float (&minus_mean)[E], const float (&rstd)[E], const float (&gamma)[E], const float (&beta)[E]) {
    float z[E];
    add_v(v, minus_mean, v);
    mul_v(v, rstd, v);
    if constexpr (ACT != kActNone) {
        fma_v(v, gamma, beta, z);
        act_slope<T, ACT>(z);
        mul_v(g, z, g);
    }
}
// dx from xhat and u, in u: rstd (u gamma - m1 - xhat m2), m1 and m2 given negated.
template <int E>
__device__ __forceinline__ void gn_dx(const float (&xhat)[E], float (&u)[E], const float (&rstd)[E], const float (&gamma)[E], const float (&minus_m1)[E], const float (&minus_m2)[E]) {
    fma_v(u, gamma, minus_m1, u);
    fma_v(xhat, minus_m2, u, u);
    mul_v(u, rstd, u);
}
// Sums of deviations from K and of their squares.
template <int E> __device__ __forceinline__ void gn_deviate(const float (&v)[E], const float (&minus_K)[E], float (&s1)[E], float (&s2)[E]) {
    float d[E];
    add_v(v, minus_K, d);
    add_v(s1, d, s1);
    fma_v(d, d, s2, s2);
}

// ------------------------------------------------------------ the CTA's cut --
// T threads as row lanes x channel chunks: chunk columns of one pass, lanes,
// and this thread's place. Where a row has more chunks than the CTA threads
// (C > E threads) the CTA takes the row in tiles of `cols` chunks.
struct Cut {
    int cols, lanes, lane, col;
    bool in;
    __device__ __forceinline__ Cut(int chunks_in_row) {
        cols = chunks_in_row < (int)blockDim.x ? chunks_in_row : (int)blockDim.x;
        lanes = (int)blockDim.x / cols;
        lane = (int)threadIdx.x / cols;
        col = (int)threadIdx.x - lane * cols;
        in = lane < lanes;
    }
};

// x of E channels, from its rows or from what they are kept as.
template <typename T, int E, bool KEPT> struct XLoad {
    typename std::conditional<KEPT, Kept<E>, Vals<T, E>>::type c;
    __device__ __forceinline__ void load(const GnParams &p, int64_t row, int ch) {
        if constexpr (KEPT)
            c.load(p.codes_in, p.scales_in, row, p.C, ch);
        else
            c.load(static_cast<const T *>(p.x) + row * p.C + ch);
    }
};

// ----------------------------------------------------------------- the flow --
// Samples that no cluster holds: one launch of persistent CTAs that take
// pieces (rows of a sample) by ticket, first to sum them and, `lag` pieces
// behind the sample's last sum, to normalise them. By then the piece's sample
// is summed and its rows still lie in the L2, so memory reads them once, and
// reads and writes overlap all the way. A piece waits only for pieces with
// earlier tickets, which running CTAs have taken and which wait for none:
// the launch makes progress however few of its CTAs run at once.
//
// A piece's group statistics, (mean, sum of squared deviations) or the two
// sums of the gradient, go to memory; the CTA that brings a sample's last
// ones joins them, in the pieces' order.

struct FlowParams {
    GnParams g;
    int pieces, lag;     // of a sample; S and A tickets of a piece lie pieces + lag pairs apart
    int64_t tickets;
    uint32_t *state;     // [0], [1]: the next ticket (64 bits); then [B] pieces summed, [B] samples joined. Zeros at the start
    float2 *part;        // [B, pieces, G]
    float2 *stat;        // [B, G]: (-mean, rstd), or the negated means of u gamma and of u gamma xhat
    int *status;
};

constexpr int kFlowThreads = 256;
constexpr uint32_t kFlowWaitLimit = 1u << 22;  // polls of 100 ns for a sample's statistics

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t *p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_release(uint32_t *p, uint32_t v) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

struct FlowShared {
    unsigned long long ticket;
    uint32_t before;
};

// The CTA's next ticket.
__device__ __forceinline__ int64_t next_ticket(const FlowParams &p, FlowShared &s) {
    __syncthreads();  // everybody is done with the last one
    if (threadIdx.x == 0) s.ticket = atomicAdd(reinterpret_cast<unsigned long long *>(p.state), 1ull);
    __syncthreads();
    return (int64_t)s.ticket;
}

// Joins a sample's pieces where this CTA's was the last: `join(g, sub, subs)`
// by `subs` neighbouring lanes a group.
template <class Join> __device__ __forceinline__ void sum_given(const FlowParams &p, FlowShared &s, int b, Join &&join) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) s.before = atomicAdd(p.state + 2 + b, 1u);
    __syncthreads();
    if (s.before != (uint32_t)p.pieces - 1) return;
    __threadfence();
    constexpr int subs = 8;
    for (int g = threadIdx.x / subs; g < (p.g.G + kFlowThreads / subs - 1) / (kFlowThreads / subs) * (kFlowThreads / subs); g += kFlowThreads / subs)
        join(g, (int)threadIdx.x % subs, subs);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) st_release(p.state + 2 + p.g.B + b, 1u);
}
__device__ __forceinline__ void wait_joined(const FlowParams &p, int b) {
    if (threadIdx.x == 0) {
        uint32_t k = 0;
        while (ld_acquire(p.state + 2 + p.g.B + b) == 0 && ++k < kFlowWaitLimit) __nanosleep(100);
        if (k >= kFlowWaitLimit && p.status) *p.status = 1;
    }
    __syncthreads();
}
template <int subs> __device__ __forceinline__ float sub_sum(float v) {
#pragma unroll
    for (int o = subs / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A thread's sums of (x - K) and (x - K)^2 a channel as mean and sum of
// squared deviations. K is its first value, so a mean far from zero costs no
// digits: the error of its sum of squares is at most n 2^-24 of it.
template <int E> __device__ __forceinline__ void lane_stats(int n, const float (&minus_K)[E], const float (&s1)[E], const float (&s2)[E], float *mean, float *m2) {
    const float inv = n > 0 ? 1.f / (float)n : 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const float m = s1[i] * inv;
        mean[i] = m - minus_K[i];
        m2[i] = fmaxf(s2[i] - s1[i] * m, 0.f);
    }
}
// The lanes' statistics of each of `width` channels ([lanes, width]) joined
// about their common mean, in place of lane 0's; `rows` in all.
__device__ __forceinline__ void join_lanes(float *mean, float *m2, int width, int lanes, int rows) {
    const int used = min(lanes, rows);
    const float all = 1.f / (float)max(rows, 1);
    for (int c = threadIdx.x; c < width; c += blockDim.x) {
        const float ref = mean[c];
        float s = 0.f, q = 0.f;
#pragma unroll 4
        for (int l = 1; l < used; ++l) s += (float)((rows - l + lanes - 1) / lanes) * (mean[l * width + c] - ref);
        const float m = ref + s * all;
#pragma unroll 4
        for (int l = 0; l < used; ++l) {
            const float d = mean[l * width + c] - m;
            q += fmaf((float)((rows - l + lanes - 1) / lanes) * d, d, m2[l * width + c]);
        }
        mean[c] = m;
        m2[c] = q;
    }
}

template <typename T, int E, int ACT, bool KEEP>
__global__ void __launch_bounds__(kFlowThreads, 2) gn_fwd_flow(const FlowParams p) {
    extern __shared__ float sm[];
    __shared__ FlowShared fs;
    float *lane_mean = sm, *lane_m2 = sm + kFlowThreads * E;
    float2 *acc = reinterpret_cast<float2 *>(sm + 2 * kFlowThreads * E);  // [G]: groups over several tiles; then the statistics
    const GnParams &g = p.g;
    pdl_wait();
    pdl_trigger();
    const int CC = g.C / E;
    const Cut cut(CC);
    const int64_t all = (int64_t)g.B * p.pieces;
    for (;;) {
        const int64_t ticket = next_ticket(p, fs);
        if (ticket >= p.tickets) return;
        const bool normalise = ticket & 1;
        const int64_t item = (ticket >> 1) - (normalise ? p.pieces + p.lag : 0);
        if (item < 0 || item >= all) continue;
        const int b = (int)(item / p.pieces), piece = (int)(item - (int64_t)b * p.pieces);
        const int64_t r0 = (int64_t)piece * g.rows, first = (int64_t)b * g.S + r0;
        const int rows = (int)min((int64_t)g.rows, g.S - r0);
        const T *x = static_cast<const T *>(g.x) + first * g.C;
        const int64_t step = (int64_t)cut.lanes * g.C;
        if (!normalise) {
            for (int t0 = 0; t0 < CC; t0 += cut.cols) {
                const int cc = t0 + cut.col;
                const int n = cut.in && cc < CC && cut.lane < rows ? (rows - cut.lane + cut.lanes - 1) / cut.lanes : 0;
                float K[E], s1[E], s2[E];
                fill_v(0.f, K);
                fill_v(0.f, s1);
                fill_v(0.f, s2);
                const T *px = x + (int64_t)cut.lane * g.C + cc * E;
                if (n > 0) {
                    Vals<T, E> c;
                    c.load(px);
                    c.get(K);
#pragma unroll
                    for (int i = 0; i < E; ++i) K[i] = -K[i];
                }
                constexpr int BATCH = 8;
                int k = 1;
                for (; k + BATCH <= n; k += BATCH) {
                    Vals<T, E> c[BATCH];
#pragma unroll
                    for (int q = 0; q < BATCH; ++q) c[q].load(px + (k + q) * step);
#pragma unroll
                    for (int q = 0; q < BATCH; ++q) {
                        float v[E];
                        c[q].get(v);
                        gn_deviate(v, K, s1, s2);
                    }
                }
#pragma unroll 4
                for (; k < n; ++k) {
                    Vals<T, E> c;
                    c.load(px + k * step);
                    float v[E];
                    c.get(v);
                    gn_deviate(v, K, s1, s2);
                }
                lane_stats(n, K, s1, s2, lane_mean + threadIdx.x * E, lane_m2 + threadIdx.x * E);
                __syncthreads();
                join_lanes(lane_mean, lane_m2, cut.cols * E, cut.lanes, rows);
                __syncthreads();
                // a warp a group: this tile's channels, joined with the tiles before
                const int c0 = t0 * E, c1 = min((t0 + cut.cols) * E, g.C);
                const int warp = threadIdx.x >> 5, wl = threadIdx.x & 31;
                for (int k2 = c0 / g.cg + warp; k2 * g.cg < c1; k2 += kFlowThreads / 32) {
                    const int lo = max(k2 * g.cg, c0), w = min((k2 + 1) * g.cg, c1) - lo;
                    const float *cm = lane_mean + (lo - c0), *cq = lane_m2 + (lo - c0);
                    const float ref = cm[0];
                    float s = 0.f, m2 = 0.f;
                    for (int c = wl; c < w; c += 32) s += cm[c] - ref;
                    s = sub_sum<32>(s);
                    float m = ref + s / (float)w;
                    for (int c = wl; c < w; c += 32) {
                        const float d = cm[c] - m;
                        m2 += fmaf((float)rows * d, d, cq[c]);
                    }
                    m2 = sub_sum<32>(m2);
                    if (wl == 0) {
                        const float cnt = (float)rows * (float)w;
                        if (lo > k2 * g.cg) {
                            const float2 a = acc[k2];
                            const float na = (float)rows * (float)(lo - k2 * g.cg), d = m - a.x, share = cnt / (na + cnt);
                            m = a.x + d * share;
                            m2 = a.y + m2 + d * d * (na * share);
                        }
                        if (lo + w < (k2 + 1) * g.cg)
                            acc[k2] = make_float2(m, m2);
                        else
                            p.part[item * g.G + k2] = make_float2(m, m2);
                    }
                }
                __syncthreads();
            }
            sum_given(p, fs, b, [&](int k, int sub, int subs) {
                const bool in = k < g.G;
                const float2 *part = p.part + (int64_t)b * p.pieces * g.G + k;
                const float n = (float)g.S * (float)g.cg;
                auto count = [&](int i) { return (float)min((int64_t)g.rows, g.S - (int64_t)i * g.rows) * (float)g.cg; };
                const float ref = in ? __ldcg(part).x : 0.f;
                float s = 0.f, m2 = 0.f;
                if (in) {
#pragma unroll 8
                    for (int i = sub; i < p.pieces; i += subs) s += count(i) * (__ldcg(part + (int64_t)i * g.G).x - ref);
                }
                const float m = ref + sub_sum<8>(s) / n;
                if (in) {
#pragma unroll 8
                    for (int i = sub; i < p.pieces; i += subs) {
                        const float2 a = __ldcg(part + (int64_t)i * g.G);
                        const float d = a.x - m;
                        m2 += fmaf(count(i) * d, d, a.y);
                    }
                }
                m2 = sub_sum<8>(m2);
                if (in && sub == 0) {
                    const float r = 1.f / sqrtf(m2 / n + g.eps);
                    p.stat[(int64_t)b * g.G + k] = make_float2(-m, r);
                    g.mean[(int64_t)b * g.G + k] = m;
                    g.rstd[(int64_t)b * g.G + k] = r;
                }
            });
            continue;
        }
        wait_joined(p, b);
        for (int k = threadIdx.x; k < g.G; k += kFlowThreads) acc[k] = __ldcg(p.stat + (int64_t)b * g.G + k);
        __syncthreads();
        T *y = static_cast<T *>(g.out) + first * g.C;
        for (int t0 = 0; t0 < CC; t0 += cut.cols) {
            const int cc = t0 + cut.col;
            if (!cut.in || cc >= CC) continue;
            float minus_mean[E], f[E], gamma[E], beta[E];
            groups_v(acc, cc * E, g.cg, g.magic, minus_mean, f);
            params_v<T>(g.gamma, g.w32, cc * E, 1.f, gamma);
            params_v<T>(g.beta, g.w32, cc * E, 0.f, beta);
            mul_v(f, gamma, f);
            constexpr int BATCH = 4;
            for (int r = cut.lane; r < rows; r += BATCH * cut.lanes) {
                Vals<T, E> c[BATCH];
#pragma unroll
                for (int q = 0; q < BATCH; ++q)
                    if (r + q * cut.lanes < rows) c[q].load_last(x + (int64_t)(r + q * cut.lanes) * g.C + cc * E);
#pragma unroll
                for (int q = 0; q < BATCH; ++q) {
                    const int rr = r + q * cut.lanes;
                    if (rr < rows) {
                        float v[E], z[E];
                        c[q].get(v);
                        gn_value<T, ACT>(v, minus_mean, f, beta, z);
                        Vals<T, E> o;
                        o.set(z);
                        o.store(y + (int64_t)rr * g.C + cc * E);
                        if constexpr (KEEP)
                            keep_chunk<T>(c[q].w, true, block_lanes<T>(), g.codes + (first + rr) * g.C + cc * E,
                                             g.scales + (first + rr) * (g.C / kBlock8) + cc * E / kBlock8);
                    }
                }
            }
        }
    }
}

template <typename T, int E, int ACT, bool KEPT>
__global__ void __launch_bounds__(kFlowThreads, 2) gn_bwd_flow(const FlowParams p) {
    extern __shared__ float sm[];
    __shared__ FlowShared fs;
    float *lane_a = sm, *lane_s = sm + kFlowThreads * E;
    float2 *acc = reinterpret_cast<float2 *>(sm + 2 * kFlowThreads * E);  // [G]
    const GnParams &g = p.g;
    pdl_wait();
    pdl_trigger();
    const int CC = g.C / E;
    const Cut cut(CC);
    const int64_t all = (int64_t)g.B * p.pieces;
    constexpr int BATCH = 4;
    for (;;) {
        const int64_t ticket = next_ticket(p, fs);
        if (ticket >= p.tickets) return;
        const bool normalise = ticket & 1;
        const int64_t item = (ticket >> 1) - (normalise ? p.pieces + p.lag : 0);
        if (item < 0 || item >= all) continue;
        const int b = (int)(item / p.pieces), piece = (int)(item - (int64_t)b * p.pieces);
        const int64_t r0 = (int64_t)piece * g.rows, first = (int64_t)b * g.S + r0;
        const int rows = (int)min((int64_t)g.rows, g.S - r0);
        const T *dy = static_cast<const T *>(g.dy) + first * g.C;
        auto constants = [&](int cc, float (&minus_mean)[E], float (&rstd)[E], float (&gamma)[E], float (&beta)[E]) {
            const int64_t at = (int64_t)b * g.G;
            auto group = [&](int c) { return g.magic ? (int)__umulhi((uint32_t)c, g.magic) : c; };
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int k = group(cc * E + i);
                minus_mean[i] = -g.mean[at + k];
                rstd[i] = g.rstd[at + k];
            }
            params_v<T>(g.gamma, g.w32, cc * E, 1.f, gamma);
            params_v<T>(g.beta, g.w32, cc * E, 0.f, beta);
        };
        if (!normalise) {
            float *out = g.parts ? g.parts + item * 2 * g.C : nullptr;
            for (int t0 = 0; t0 < CC; t0 += cut.cols) {
                const int cc = t0 + cut.col;
                float a[E], s[E];
                fill_v(0.f, a);
                fill_v(0.f, s);
                if (cut.in && cc < CC) {
                    float minus_mean[E], rstd[E], gamma[E], beta[E];
                    constants(cc, minus_mean, rstd, gamma, beta);
                    for (int r = cut.lane; r < rows; r += BATCH * cut.lanes) {
                        XLoad<T, E, KEPT> x[BATCH];
                        Vals<T, E> d[BATCH];
#pragma unroll
                        for (int q = 0; q < BATCH; ++q) {
                            const int rr = r + q * cut.lanes;
                            if (rr < rows) {
                                x[q].load(g, first + rr, cc * E);
                                d[q].load(dy + (int64_t)rr * g.C + cc * E);
                            }
                        }
#pragma unroll
                        for (int q = 0; q < BATCH; ++q)
                            if (r + q * cut.lanes < rows) {
                                float v[E], u[E];
                                x[q].c.get(v);
                                d[q].get(u);
                                gn_slope<T, ACT>(v, u, minus_mean, rstd, gamma, beta);
                                fma_v(u, v, a, a);
                                add_v(s, u, s);
                            }
                    }
                }
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    lane_a[threadIdx.x * E + i] = a[i];
                    lane_s[threadIdx.x * E + i] = s[i];
                }
                __syncthreads();
                const int width = cut.cols * E, c0 = t0 * E, c1 = min(c0 + width, g.C);
                for (int c = threadIdx.x; c < c1 - c0; c += kFlowThreads) {
                    float ta = lane_a[c], ts = lane_s[c];
#pragma unroll 4
                    for (int l = 1; l < cut.lanes; ++l) {
                        ta += lane_a[l * width + c];
                        ts += lane_s[l * width + c];
                    }
                    if (out) {
                        out[c0 + c] = ta;
                        out[g.C + c0 + c] = ts;
                    }
                    const float ga = param<T>(g.gamma, g.w32, c0 + c, 1.f);
                    lane_a[c] = ta * ga;
                    lane_s[c] = ts * ga;
                }
                __syncthreads();
                const int warp = threadIdx.x >> 5, wl = threadIdx.x & 31;
                for (int k = c0 / g.cg + warp; k * g.cg < c1; k += kFlowThreads / 32) {
                    const int lo = max(k * g.cg, c0), hi = min((k + 1) * g.cg, c1);
                    float2 m = make_float2(0.f, 0.f);
                    for (int c = lo + wl; c < hi; c += 32) m = add2(m, make_float2(lane_s[c - c0], lane_a[c - c0]));
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) m = add2(m, shfl_xor2(m, o));
                    if (wl == 0) {
                        if (lo > k * g.cg) m = add2(acc[k], m);
                        if (hi < (k + 1) * g.cg)
                            acc[k] = m;
                        else
                            p.part[item * g.G + k] = m;
                    }
                }
                __syncthreads();
            }
            sum_given(p, fs, b, [&](int k, int sub, int subs) {
                const bool in = k < g.G;
                const float2 *part = p.part + (int64_t)b * p.pieces * g.G + k;
                float2 m = make_float2(0.f, 0.f);
                if (in) {
#pragma unroll 8
                    for (int i = sub; i < p.pieces; i += subs) m = add2(m, __ldcg(part + (int64_t)i * g.G));
                }
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) m = add2(m, shfl_xor2(m, o));
                const float n = (float)g.S * (float)g.cg;
                if (in && sub == 0) p.stat[(int64_t)b * g.G + k] = make_float2(-m.x / n, -m.y / n);
            });
            continue;
        }
        wait_joined(p, b);
        for (int k = threadIdx.x; k < g.G; k += kFlowThreads) acc[k] = __ldcg(p.stat + (int64_t)b * g.G + k);
        __syncthreads();
        T *dx = static_cast<T *>(g.out) + first * g.C;
        for (int t0 = 0; t0 < CC; t0 += cut.cols) {
            const int cc = t0 + cut.col;
            if (!cut.in || cc >= CC) continue;
            float minus_mean[E], rstd[E], gamma[E], beta[E], m1[E], m2[E];
            constants(cc, minus_mean, rstd, gamma, beta);
            groups_v(acc, cc * E, g.cg, g.magic, m1, m2);
            constexpr int HALF = 2;
            for (int r = cut.lane; r < rows; r += HALF * cut.lanes) {
                XLoad<T, E, KEPT> x[HALF];
                Vals<T, E> d[HALF];
#pragma unroll
                for (int q = 0; q < HALF; ++q) {
                    const int rr = r + q * cut.lanes;
                    if (rr < rows) {
                        x[q].load(g, first + rr, cc * E);
                        d[q].load_last(dy + (int64_t)rr * g.C + cc * E);
                    }
                }
#pragma unroll
                for (int q = 0; q < HALF; ++q) {
                    const int rr = r + q * cut.lanes;
                    if (rr < rows) {
                        float v[E], u[E];
                        x[q].c.get(v);
                        d[q].get(u);
                        gn_slope<T, ACT>(v, u, minus_mean, rstd, gamma, beta);
                        gn_dx(v, u, rstd, gamma, m1, m2);
                        Vals<T, E> o;
                        o.set(u);
                        o.store(dx + (int64_t)rr * g.C + cc * E);
                    }
                }
            }
        }
    }
}

// Many rows of sums folded into gridDim.y: row i of the result is the sum of
// rows [i n / gridDim.y, (i + 1) n / gridDim.y), in order.
static __global__ void __launch_bounds__(256) gn_fold(const float *in, float *out, int64_t n, int width) {
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x * 256 + threadIdx.x;
    const int64_t i0 = n * blockIdx.y / gridDim.y, i1 = n * (blockIdx.y + 1) / gridDim.y;
    if (c >= width) return;
    float s = 0.f;
#pragma unroll 8
    for (int64_t i = i0; i < i1; ++i) s += in[i * width + c];
    out[(int64_t)blockIdx.y * width + c] = s;
}

// ---------------------------------------------------------------- kernels --

// (keeping x in the same pass: whole 16-byte chunks only)
template <typename T, int E, int ACT> static const void *gn_flow_fwd(bool kept) {
    if constexpr (E > 1) {
        if (kept) return (const void *)gn_fwd_flow<T, E, ACT, true>;
    }
    return (const void *)gn_fwd_flow<T, E, ACT, false>;
}
template <typename T, int E> static const void *gn_flow_e(bool backward, int act, bool kept) {
#define FLOW(A)                                                                                              \
    (!backward ? gn_flow_fwd<T, E, A>(kept)                                                                  \
     : kept    ? (const void *)gn_bwd_flow<T, E, A, true>                                                    \
               : (const void *)gn_bwd_flow<T, E, A, false>)
    return act == kActSilu ? FLOW(kActSilu) : act == kActGelu ? FLOW(kActGelu) : FLOW(kActNone);
#undef FLOW
}
// A kernel by 16-byte chunks (wide) or by single values.
template <typename T> static const void *gn_flow_t(bool backward, bool wide, int act, bool kept) {
    return wide ? gn_flow_e<T, Elem<T>::E>(backward, act, kept) : gn_flow_e<T, 1>(backward, act, kept);
}

#define GN_DECLARE(suf)                                                          \
    const void *gn_flow_##suf(bool backward, bool wide, int act, bool kept);     \
    const void *gn_held_##suf(bool backward, bool wide, int act, bool kept);
GN_DECLARE(f32)
GN_DECLARE(bf16)
GN_DECLARE(f16)
#undef GN_DECLARE

}  // namespace rmsn
