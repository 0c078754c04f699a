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
    float *parts;              // a chunk's sums: [B, chunks, G, 2] (forward), [B, chunks, 2, C] (backward)
    float *sums;               // backward: [B, 2, C], a sample's sums of u xhat and of u
    float2 *means;             // backward: [B, G], the group means of u gamma and of u gamma xhat
    int64_t S;
    int B, C, G, cg;           // cg = C / G
    int b0;                    // first sample of the launch
    int rows, chunks;          // rows a CTA takes, CTAs a sample
    int act, w32;
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

// ------------------------------------------------------------- activations --
// The sigmoids of two values. For 16-bit rows one reciprocal serves both
// (1 / a = b / (a b)): the special-function unit, 16 results a clock and SM,
// bounds these kernels next to memory, and so it gives 1.5 results a value
// instead of 2. z is held at -43, where the sigmoid is 2^-62 and a b still
// finite. fp32 rows take the accurate exponential.
template <typename T> __device__ __forceinline__ float2 sigmoid2(float2 z) {
    if constexpr (std::is_same<T, float>::value) {
        return make_float2(__fdividef(1.f, 1.f + expf(-z.x)), __fdividef(1.f, 1.f + expf(-z.y)));
    } else {
        const float a = 1.f + __expf(-fmaxf(z.x, -43.f)), b = 1.f + __expf(-fmaxf(z.y, -43.f));
        const float r = __fdividef(1.f, a * b);
        return make_float2(r * b, r * a);
    }
}
template <typename T> __device__ __forceinline__ float sigmoid(float z) {
    if constexpr (std::is_same<T, float>::value)
        return __fdividef(1.f, 1.f + expf(-z));
    else
        return __fdividef(1.f, 1.f + __expf(-fmaxf(z, -43.f)));
}
// (fmaxf drops a NaN: z, which every result is multiplied by, brings it back.)

__device__ __forceinline__ float gelu_of(float z) { return 0.5f * z * (1.f + erff(z * 0.70710678f)); }
__device__ __forceinline__ float gelu_slope(float z) {
    return 0.5f * (1.f + erff(z * 0.70710678f)) + z * __expf(-0.5f * z * z) * 0.39894228f;
}

// act(z) and act'(z) of E values, in place.
template <typename T, int ACT, int E> __device__ __forceinline__ void act_of(float (&z)[E]) {
    if constexpr (ACT == kActSilu) {
        if constexpr (E > 1) {
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                const float2 p = sigmoid2<T>(make_float2(z[i], z[i + 1]));
                z[i] *= p.x, z[i + 1] *= p.y;
            }
        } else {
            z[0] *= sigmoid<T>(z[0]);
        }
    } else if constexpr (ACT == kActGelu) {
#pragma unroll
        for (int i = 0; i < E; ++i) z[i] = gelu_of(z[i]);
    }
}
template <typename T, int ACT, int E> __device__ __forceinline__ void act_slope(float (&z)[E]) {
    if constexpr (ACT == kActSilu) {
        float p[E];
        if constexpr (E > 1) {
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                const float2 q = sigmoid2<T>(make_float2(z[i], z[i + 1]));
                p[i] = q.x, p[i + 1] = q.y;
            }
        } else {
            p[0] = sigmoid<T>(z[0]);
        }
#pragma unroll
        for (int i = 0; i < E; ++i) z[i] = p[i] * fmaf(z[i], 1.f - p[i], 1.f);
    } else if constexpr (ACT == kActGelu) {
#pragma unroll
        for (int i = 0; i < E; ++i) z[i] = gelu_slope(z[i]);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) z[i] = 1.f;
    }
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

constexpr int kGnBatch = 4;  // rows of a thread under way at once

// ----------------------------------------------------------------- forward --
// A chunk of rows' statistics, (mean, sum of squared deviations) for each
// group. A thread sums (x - K) and (x - K)^2 a channel, K its first value, so
// a mean far from zero costs no digits: the error of its sum of squares is at
// most rows 2^-24 of it, whatever K is, and the pieces are then joined about
// their own means.
template <typename T, int E>
__global__ void __launch_bounds__(512) gn_stats(const GnParams p) {
    extern __shared__ float sm[];
    float *sm_mean = sm, *sm_m2 = sm + blockDim.x * E;
    float2 *acc = reinterpret_cast<float2 *>(sm + 2 * blockDim.x * E);  // [G], (mean, M2) over the tiles so far
    pdl_wait();
    pdl_trigger();
    const int b = p.b0 + blockIdx.y;
    const int64_t r0 = (int64_t)blockIdx.x * p.rows;
    const int rows = (int)min((int64_t)p.rows, p.S - r0);
    const int CC = p.C / E;
    const Cut cut(CC);
    const T *x = static_cast<const T *>(p.x) + ((int64_t)b * p.S + r0) * p.C;
    for (int t0 = 0; t0 < CC; t0 += cut.cols) {
        const int cc = t0 + cut.col;
        const int n = cut.in && cc < CC && cut.lane < rows ? (rows - cut.lane + cut.lanes - 1) / cut.lanes : 0;
        float K[E], s1[E], s2[E];
#pragma unroll
        for (int i = 0; i < E; ++i) K[i] = s1[i] = s2[i] = 0.f;
        const T *px = x + (int64_t)cut.lane * p.C + (int64_t)cc * E;
        const int64_t step = (int64_t)cut.lanes * p.C;
        for (int k = 0; k < n; k += kGnBatch) {
            Vals<T, E> c[kGnBatch];
#pragma unroll
            for (int q = 0; q < kGnBatch; ++q)
                if (k + q < n) c[q].load(px + (k + q) * step);
#pragma unroll
            for (int q = 0; q < kGnBatch; ++q)
                if (k + q < n) {
                    float v[E];
                    c[q].get(v);
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        if (k + q == 0) K[i] = v[i];
                        const float d = v[i] - K[i];
                        s1[i] += d;
                        s2[i] = fmaf(d, d, s2[i]);
                    }
                }
        }
        const float inv = n > 0 ? 1.f / (float)n : 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float m = s1[i] * inv;
            sm_mean[threadIdx.x * E + i] = K[i] + m;
            sm_m2[threadIdx.x * E + i] = fmaxf(s2[i] - s1[i] * m, 0.f);
        }
        __syncthreads();
        // a warp a group: the lanes' and channels' pieces of this tile, then joined with the tiles before
        const int c0 = t0 * E, c1 = min((t0 + cut.cols) * E, p.C);
        const int warp = threadIdx.x >> 5, wl = threadIdx.x & 31;
        const int width = cut.cols * E;
        for (int g = c0 / p.cg + warp; g * p.cg < c1; g += blockDim.x >> 5) {
            const int lo = max(g * p.cg, c0), w = min((g + 1) * p.cg, c1) - lo;
            const int used = min(cut.lanes, rows);  // lanes with rows
            const float *mean0 = sm_mean + (lo - c0), *m20 = sm_m2 + (lo - c0);
            const float ref = mean0[0];
            float s = 0.f;
            for (int i = wl; i < used * w; i += 32) {
                const int l = i / w, c = i - l * w;
                s += (float)((rows - l + cut.lanes - 1) / cut.lanes) * (mean0[l * width + c] - ref);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            const float cnt = (float)rows * (float)w;
            float m = ref + s / cnt, m2 = 0.f;
            for (int i = wl; i < used * w; i += 32) {
                const int l = i / w, c = i - l * w;
                const float d = mean0[l * width + c] - m;
                m2 += fmaf((float)((rows - l + cut.lanes - 1) / cut.lanes) * d, d, m20[l * width + c]);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m2 += __shfl_xor_sync(0xffffffffu, m2, o);
            if (wl == 0) {
                if (lo > g * p.cg) {  // the group's first channels were in earlier tiles
                    const float2 a = acc[g];
                    const float na = (float)rows * (float)(lo - g * p.cg), all = na + cnt, d = m - a.x;
                    m = a.x + d * (cnt / all);
                    m2 = a.y + m2 + d * d * (na * (cnt / all));
                }
                if (lo + w < (g + 1) * p.cg)
                    acc[g] = make_float2(m, m2);
                else
                    reinterpret_cast<float2 *>(p.parts)[((int64_t)b * p.chunks + blockIdx.x) * p.G + g] = make_float2(m, m2);
            }
        }
        __syncthreads();
    }
}

// A sample's statistics from its chunks', into shared memory (every CTA of
// the sample joins them anew, in one order: all have the same bits).
__device__ __forceinline__ void gn_join(const GnParams &p, int b, float2 *stat, bool write) {
    const int warp = threadIdx.x >> 5, wl = threadIdx.x & 31;
    for (int g = warp; g < p.G; g += blockDim.x >> 5) {
        const float2 *part = reinterpret_cast<const float2 *>(p.parts) + (int64_t)b * p.chunks * p.G + g;
        const float ref = part[0].x;
        const float n = (float)p.S * (float)p.cg;
        auto count = [&](int i) { return (float)min((int64_t)p.rows, p.S - (int64_t)i * p.rows) * (float)p.cg; };
        float s = 0.f;
        for (int i = wl; i < p.chunks; i += 32) s += count(i) * (part[(int64_t)i * p.G].x - ref);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const float m = ref + s / n;
        float m2 = 0.f;
        for (int i = wl; i < p.chunks; i += 32) {
            const float2 a = part[(int64_t)i * p.G];
            const float d = a.x - m;
            m2 += fmaf(count(i) * d, d, a.y);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m2 += __shfl_xor_sync(0xffffffffu, m2, o);
        if (wl == 0) {
            const float r = 1.f / sqrtf(m2 / n + p.eps);
            stat[g] = make_float2(m, r);
            if (write) {
                p.mean[(int64_t)b * p.G + g] = m;
                p.rstd[(int64_t)b * p.G + g] = r;
            }
        }
    }
}

template <typename T, int E, int ACT, bool KEEP>
__global__ void __launch_bounds__(512) gn_apply(const GnParams p) {
    extern __shared__ float sm[];
    float2 *stat = reinterpret_cast<float2 *>(sm);
    pdl_wait();
    pdl_trigger();
    const int b = p.b0 + blockIdx.y;
    const int64_t r0 = (int64_t)blockIdx.x * p.rows;
    const int rows = (int)min((int64_t)p.rows, p.S - r0);
    const int CC = p.C / E;
    const Cut cut(CC);
    gn_join(p, b, stat, blockIdx.x == 0);
    __syncthreads();
    const int64_t at = ((int64_t)b * p.S + r0) * p.C;
    const T *x = static_cast<const T *>(p.x) + at;
    T *y = static_cast<T *>(p.out) + at;
    for (int t0 = 0; t0 < CC; t0 += cut.cols) {
        const int cc = t0 + cut.col;
        if (!cut.in || cc >= CC) continue;
        float mean[E], f[E], beta[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = cc * E + i;
            const float2 s = stat[c / p.cg];
            mean[i] = s.x;
            f[i] = s.y * param<T>(p.gamma, p.w32, c, 1.f);
            beta[i] = param<T>(p.beta, p.w32, c, 0.f);
        }
        for (int r = cut.lane; r < rows; r += kGnBatch * cut.lanes) {
            Vals<T, E> c[kGnBatch];
#pragma unroll
            for (int q = 0; q < kGnBatch; ++q)
                if (r + q * cut.lanes < rows) c[q].load_last(x + (int64_t)(r + q * cut.lanes) * p.C + cc * E);
#pragma unroll
            for (int q = 0; q < kGnBatch; ++q) {
                const int rr = r + q * cut.lanes;
                if (rr < rows) {
                    float v[E], z[E];
                    c[q].get(v);
#pragma unroll
                    for (int i = 0; i < E; ++i) z[i] = fmaf(v[i] - mean[i], f[i], beta[i]);
                    act_of<T, ACT>(z);
                    Vals<T, E> o;
                    o.set(z);
                    o.store(y + (int64_t)rr * p.C + cc * E);
                    if constexpr (KEEP) {
                        const int64_t row = (int64_t)b * p.S + r0 + rr;
                        keep_chunk<T, E>(v, true, p.codes + row * p.C + cc * E, p.scales + row * (p.C / kBlock8) + cc * E / kBlock8);
                    }
                }
            }
        }
    }
}

// ---------------------------------------------------------------- backward --

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

// A chunk of rows' sums of u xhat and of u for each channel.
template <typename T, int E, int ACT, bool KEPT>
__global__ void __launch_bounds__(256) gn_bwd_sums(const GnParams p) {
    extern __shared__ float sm[];
    float *sa = sm, *sb = sm + blockDim.x * E;
    pdl_wait();
    pdl_trigger();
    const int b = p.b0 + blockIdx.y;
    const int64_t r0 = (int64_t)blockIdx.x * p.rows;
    const int rows = (int)min((int64_t)p.rows, p.S - r0);
    const int64_t first = (int64_t)b * p.S + r0;
    const int CC = p.C / E;
    const Cut cut(CC);
    const T *dy = static_cast<const T *>(p.dy) + first * p.C;
    float *out = p.parts + ((int64_t)b * p.chunks + blockIdx.x) * 2 * p.C;
    for (int t0 = 0; t0 < CC; t0 += cut.cols) {
        const int cc = t0 + cut.col;
        const bool in = cut.in && cc < CC;
        float a[E], s[E];
#pragma unroll
        for (int i = 0; i < E; ++i) a[i] = s[i] = 0.f;
        if (in) {
            float mean[E], rstd[E], gamma[E], beta[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = cc * E + i;
                mean[i] = p.mean[(int64_t)b * p.G + c / p.cg];
                rstd[i] = p.rstd[(int64_t)b * p.G + c / p.cg];
                gamma[i] = param<T>(p.gamma, p.w32, c, 1.f);
                beta[i] = param<T>(p.beta, p.w32, c, 0.f);
            }
            for (int r = cut.lane; r < rows; r += kGnBatch * cut.lanes) {
                XLoad<T, E, KEPT> x[kGnBatch];
                Vals<T, E> d[kGnBatch];
#pragma unroll
                for (int q = 0; q < kGnBatch; ++q) {
                    const int rr = r + q * cut.lanes;
                    if (rr < rows) {
                        x[q].load(p, first + rr, cc * E);
                        d[q].load(dy + (int64_t)rr * p.C + cc * E);
                    }
                }
#pragma unroll
                for (int q = 0; q < kGnBatch; ++q)
                    if (r + q * cut.lanes < rows) {
                        float v[E], g[E], z[E];
                        x[q].c.get(v);
                        d[q].get(g);
#pragma unroll
                        for (int i = 0; i < E; ++i) {
                            v[i] = (v[i] - mean[i]) * rstd[i];
                            z[i] = fmaf(v[i], gamma[i], beta[i]);
                        }
                        act_slope<T, ACT>(z);
#pragma unroll
                        for (int i = 0; i < E; ++i) {
                            const float u = g[i] * z[i];
                            a[i] = fmaf(u, v[i], a[i]);
                            s[i] += u;
                        }
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
            sa[threadIdx.x * E + i] = a[i];
            sb[threadIdx.x * E + i] = s[i];
        }
        __syncthreads();
        const int width = cut.cols * E;
        for (int c = threadIdx.x; c < width; c += blockDim.x)
            if (t0 * E + c < p.C) {
                float ta = sa[c], ts = sb[c];
                for (int l = 1; l < cut.lanes; ++l) {
                    ta += sa[l * width + c];
                    ts += sb[l * width + c];
                }
                out[t0 * E + c] = ta;
                out[p.C + t0 * E + c] = ts;
            }
        __syncthreads();
    }
}

// A sample's sums over its chunks, in order, and its groups' means: a CTA
// takes groups [blockIdx.x gpc, ...) of sample b0 + blockIdx.y.
constexpr int kGnReduceThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kGnReduceThreads) gn_bwd_reduce(const GnParams p, int groups_a_cta) {
    __shared__ float2 red[kGnReduceThreads / 32];
    pdl_wait();
    pdl_trigger();
    const int b = p.b0 + blockIdx.y;
    const float *part = p.parts + (int64_t)b * p.chunks * 2 * p.C;
    float *sums = p.sums + (int64_t)b * 2 * p.C;
    const float n = (float)p.S * (float)p.cg;
    const int g1 = min((blockIdx.x + 1) * groups_a_cta, (unsigned)p.G);
    for (int g = blockIdx.x * groups_a_cta; g < g1; ++g) {
        float2 m = make_float2(0.f, 0.f);
        for (int c = g * p.cg + threadIdx.x; c < (g + 1) * p.cg; c += blockDim.x) {
            float a = 0.f, s = 0.f;
#pragma unroll 8
            for (int k = 0; k < p.chunks; ++k) {
                a += part[(int64_t)k * 2 * p.C + c];
                s += part[(int64_t)k * 2 * p.C + p.C + c];
            }
            sums[c] = a;
            sums[p.C + c] = s;
            const float gamma = param<T>(p.gamma, p.w32, c, 1.f);
            m.x = fmaf(s, gamma, m.x);
            m.y = fmaf(a, gamma, m.y);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = add2(m, shfl_xor2(m, o));
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
        __syncthreads();
        if (threadIdx.x == 0) {
            float2 t = red[0];
            for (int i = 1; i < (int)blockDim.x / 32; ++i) t = add2(t, red[i]);
            p.means[(int64_t)b * p.G + g] = make_float2(t.x / n, t.y / n);
        }
        __syncthreads();
    }
}

template <typename T, int E, int ACT, bool KEPT>
__global__ void __launch_bounds__(256) gn_bwd_apply(const GnParams p) {
    pdl_wait();
    pdl_trigger();
    const int b = p.b0 + blockIdx.y;
    const int64_t r0 = (int64_t)blockIdx.x * p.rows;
    const int rows = (int)min((int64_t)p.rows, p.S - r0);
    const int64_t first = (int64_t)b * p.S + r0;
    const int CC = p.C / E;
    const Cut cut(CC);
    const T *dy = static_cast<const T *>(p.dy) + first * p.C;
    T *dx = static_cast<T *>(p.out) + first * p.C;
    for (int t0 = 0; t0 < CC; t0 += cut.cols) {
        const int cc = t0 + cut.col;
        if (!cut.in || cc >= CC) continue;
        float mean[E], rstd[E], gamma[E], beta[E], m1[E], m2[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = cc * E + i;
            const int64_t g = (int64_t)b * p.G + c / p.cg;
            mean[i] = p.mean[g];
            rstd[i] = p.rstd[g];
            gamma[i] = param<T>(p.gamma, p.w32, c, 1.f);
            beta[i] = param<T>(p.beta, p.w32, c, 0.f);
            const float2 m = p.means[g];
            m1[i] = m.x;
            m2[i] = m.y;
        }
        for (int r = cut.lane; r < rows; r += kGnBatch * cut.lanes) {
            XLoad<T, E, KEPT> x[kGnBatch];
            Vals<T, E> d[kGnBatch];
#pragma unroll
            for (int q = 0; q < kGnBatch; ++q) {
                const int rr = r + q * cut.lanes;
                if (rr < rows) {
                    x[q].load(p, first + rr, cc * E);
                    d[q].load_last(dy + (int64_t)rr * p.C + cc * E);
                }
            }
#pragma unroll
            for (int q = 0; q < kGnBatch; ++q) {
                const int rr = r + q * cut.lanes;
                if (rr < rows) {
                    float v[E], g[E], z[E];
                    x[q].c.get(v);
                    d[q].get(g);
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        v[i] = (v[i] - mean[i]) * rstd[i];
                        z[i] = fmaf(v[i], gamma[i], beta[i]);
                    }
                    act_slope<T, ACT>(z);
#pragma unroll
                    for (int i = 0; i < E; ++i) g[i] = rstd[i] * (fmaf(g[i] * z[i], gamma[i], -m1[i]) - v[i] * m2[i]);
                    Vals<T, E> o;
                    o.set(g);
                    o.store(dx + (int64_t)rr * p.C + cc * E);
                }
            }
        }
    }
}

// ---------------------------------------------------------------- launches --

// Which of the compiled widths a call takes: 16-byte chunks, or one value.
enum { kGnStats = 0, kGnApply, kGnBwdSums, kGnBwdReduce, kGnBwdApply };

template <typename T, int E>
static const void *gn_kernel_e(int which, int act, bool kept) {
    switch (which) {
    case kGnStats: return (const void *)gn_stats<T, E>;
    case kGnApply:
        if constexpr (E > 1) {
            if (kept)
                return act == kActSilu   ? (const void *)gn_apply<T, E, kActSilu, true>
                       : act == kActGelu ? (const void *)gn_apply<T, E, kActGelu, true>
                                         : (const void *)gn_apply<T, E, kActNone, true>;
        }
        return act == kActSilu   ? (const void *)gn_apply<T, E, kActSilu, false>
               : act == kActGelu ? (const void *)gn_apply<T, E, kActGelu, false>
                                 : (const void *)gn_apply<T, E, kActNone, false>;
    case kGnBwdSums:
        if (kept)
            return act == kActSilu   ? (const void *)gn_bwd_sums<T, E, kActSilu, true>
                   : act == kActGelu ? (const void *)gn_bwd_sums<T, E, kActGelu, true>
                                     : (const void *)gn_bwd_sums<T, E, kActNone, true>;
        return act == kActSilu   ? (const void *)gn_bwd_sums<T, E, kActSilu, false>
               : act == kActGelu ? (const void *)gn_bwd_sums<T, E, kActGelu, false>
                                 : (const void *)gn_bwd_sums<T, E, kActNone, false>;
    case kGnBwdReduce: return (const void *)gn_bwd_reduce<T>;
    default:
        if (kept)
            return act == kActSilu   ? (const void *)gn_bwd_apply<T, E, kActSilu, true>
                   : act == kActGelu ? (const void *)gn_bwd_apply<T, E, kActGelu, true>
                                     : (const void *)gn_bwd_apply<T, E, kActNone, true>;
        return act == kActSilu   ? (const void *)gn_bwd_apply<T, E, kActSilu, false>
               : act == kActGelu ? (const void *)gn_bwd_apply<T, E, kActGelu, false>
                                 : (const void *)gn_bwd_apply<T, E, kActNone, false>;
    }
}

template <typename T> static const void *gn_kernel_t(int which, bool wide, int act, bool kept) {
    return wide ? gn_kernel_e<T, Elem<T>::E>(which, act, kept) : gn_kernel_e<T, 1>(which, act, kept);
}

const void *gn_kernel_f32(int which, bool wide, int act, bool kept);
const void *gn_kernel_bf16(int which, bool wide, int act, bool kept);
const void *gn_kernel_f16(int which, bool wide, int act, bool kept);

}  // namespace rmsn
