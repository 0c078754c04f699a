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

// Values of a chunk: 16 bytes where the channels' count and the addresses
// allow it, else 8 bytes of 16-bit rows, else single values.
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
template <typename T> __device__ __forceinline__ float2 widen2(uint32_t u);
template <> __device__ __forceinline__ float2 widen2<__nv_bfloat16>(uint32_t u) { return bf16x2_to_f2(u); }
template <> __device__ __forceinline__ float2 widen2<__half>(uint32_t u) { return f16x2_to_f2(u); }
template <typename T> __device__ __forceinline__ uint32_t narrow2(float2 v);
template <> __device__ __forceinline__ uint32_t narrow2<__nv_bfloat16>(float2 v) { return f2_to_bf16x2(v); }
template <> __device__ __forceinline__ uint32_t narrow2<__half>(float2 v) { return f2_to_f16x2(v); }

template <typename T, int E> struct Vals {
    static constexpr int B = E * (int)sizeof(T), N = B >= 4 ? B / 4 : 1;
    using W = typename Word<B>::type;
    union {
        W w;
        uint32_t u[N];
    };
    __device__ __forceinline__ Vals() {}
    __device__ __forceinline__ void load(const T *p) { w = *reinterpret_cast<const W *>(p); }
    __device__ __forceinline__ void load_last(const T *p) { w = __ldcs(reinterpret_cast<const W *>(p)); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<W *>(p) = w; }
    __device__ __forceinline__ void get(float (&v)[E]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = __uint_as_float(u[i]);
        } else if constexpr (E > 1) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const float2 q = widen2<T>(u[i]);
                v[2 * i] = q.x, v[2 * i + 1] = q.y;
            }
        } else {
            v[0] = widen<T>(*reinterpret_cast<const T *>(&w));
        }
    }
    __device__ __forceinline__ void set(const float (&v)[E]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < E; ++i) u[i] = __float_as_uint(v[i]);
        } else if constexpr (E > 1) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) u[i] = narrow2<T>(make_float2(v[2 * i], v[2 * i + 1]));
        } else {
            store_elem(reinterpret_cast<T *>(&w), 0, v[0]);
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

// The sigmoids of E values: 1 / (1 + 2^(-z log2 e)), the reciprocal and (for
// 16-bit rows) the exponential the fast ones; fp32 rows take the accurate
// exponential. (SiLU in fp32 over [-8, 8]: rms error 1.50e-7 with the fast
// reciprocal, 1.44e-7 with a division; its slope 1.11e-7 and 1.06e-7.) (One reciprocal for two values, 1 / a = b / (a b), takes 12
// instead of 16 results of the special-function unit for 8 values, but 20
// instructions more, and was no faster: 16.5 and 16.9 us for 8 x 4096 x 320.)
template <typename T, int E> __device__ __forceinline__ void sigmoid_v(const float (&z)[E], float (&p)[E]) {
    if constexpr (std::is_same<T, float>::value) {
#pragma unroll
        for (int i = 0; i < E; ++i) p[i] = rcp_fast(1.f + expf(-z[i]));
    } else {
        float k[E], one[E];
        fill_v(-1.4426950f, k);
        fill_v(1.f, one);
        mul_v(z, k, p);
#pragma unroll
        for (int i = 0; i < E; ++i) p[i] = exp2_fast(p[i]);
        add_v(p, one, p);
#pragma unroll
        for (int i = 0; i < E; ++i) p[i] = rcp_fast(p[i]);
    }
}
// GELU as 1 + erf: over [-8, 8] off by 4.9e-7 at most (8 2^-24, rms 7e-8); below
// z = -4 the digits that cancel are lost (6% of the value at -5), as in any form
// with 1 + erf in 32 bits. The slope is off by 1.4e-7 at most (rms 2.7e-8), the
// same with expf in the place of __expf.
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
// A CTA's threads as row lanes x channel chunks: chunk columns of one pass,
// lanes, and this thread's place. Where a row has more chunks than the CTA
// threads, the CTA takes it in tiles of equal width.
struct Cut {
    int cols, lanes, lane, col;
    bool in;
    __device__ __forceinline__ Cut(int chunks_in_row, int threads) {
        const int tiles = (chunks_in_row + threads - 1) / threads;
        cols = (chunks_in_row + tiles - 1) / tiles;
        if (tiles > 1) cols = (cols + 7) & ~7;  // (a block of 32 values is 8 lanes of a tile)
        lanes = threads / cols;
        lane = (int)threadIdx.x / cols;
        col = (int)threadIdx.x - lane * cols;
        in = lane < lanes;
    }
};

// A lane's rows of `rows`: lane, lane + lanes, ...
__device__ __forceinline__ int rows_of_lane(int rows, int lane, int lanes) { return lane < rows ? (rows - lane + lanes - 1) / lanes : 0; }

// ------------------------------------------------------------- statistics --
// A thread's sums of (x - K) and (x - K)^2 a channel as mean and sum of
// squared deviations. K is its first value, so a mean far from zero costs no
// digits: the error of its sum of squares is at most n 2^-24 of it.
// E floats to shared memory, 16 bytes at a time.
template <int E> __device__ __forceinline__ void put_v(float *to, const float (&v)[E]) {
    if constexpr (E % 4 == 0) {
#pragma unroll
        for (int i = 0; i < E; i += 4) *reinterpret_cast<float4 *>(to + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) to[i] = v[i];
    }
}
// A sum of squares that cancellation left below 0 is 0; a NaN stays.
__device__ __forceinline__ float at_least_0(float v) { return v < 0.f ? 0.f : v; }
template <int E> __device__ __forceinline__ void lane_stats(int n, const float (&minus_K)[E], const float (&s1)[E], const float (&s2)[E], float *mean, float *m2) {
    const float inv = n > 0 ? 1.f / (float)n : 0.f;
    float m[E], q[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        m[i] = s1[i] * inv;
        q[i] = at_least_0(s2[i] - s1[i] * m[i]);
        m[i] -= minus_K[i];
    }
    put_v(mean, m);
    put_v(m2, q);
}
// The lanes' statistics of each of `width` channels ([lanes, width]) joined in
// place of lane 0's; `rows` in all. About lane 0's mean: with 1 / lanes of the
// rows its own, it is at most sqrt(lanes) widths off the common one.
template <int THREADS> __device__ __forceinline__ void join_lanes(float *mean, float *m2, int width, int lanes, int rows) {
    const int used = min(lanes, rows), each = rows / lanes, more = rows - each * lanes;  // rows of a lane, lanes with one more
    const float few = (float)each, many = (float)(each + 1), all = 1.f / (float)max(rows, 1);
    if (lanes == 1) return;
    for (int c = threadIdx.x; c < width; c += THREADS) {
        const float ref = mean[c];
        float s = 0.f, q = m2[c];
#pragma unroll 8
        for (int l = 1; l < used; ++l) {
            const float d = mean[l * width + c] - ref, nd = (l < more ? many : few) * d;
            s += nd;
            q += fmaf(nd, d, m2[l * width + c]);
        }
        const float m = s * all;
        mean[c] = ref + m;
        m2[c] = at_least_0(q - s * m);
    }
}
// For each group with channels among [c0, c1): both values of its channels
// there summed (`each(c)` gives them), by a team of as many lanes as it has
// channels (a power of two, a warp at most). give(k, lo, hi, sums) is called by
// one lane a group.
template <int THREADS, class Each, class Give>
__device__ __forceinline__ void sum_groups(int c0, int c1, int cg, Each &&each, Give &&give) {
    int ts = 1;
    while (ts < cg && ts < 32) ts *= 2;
    const int team = (int)threadIdx.x / ts, tl = (int)threadIdx.x % ts, teams = THREADS / ts;
    for (int k0 = c0 / cg; k0 * cg < c1; k0 += teams) {
        const int k = k0 + team, lo = max(k * cg, c0), hi = min((k + 1) * cg, c1);
        float2 m = make_float2(0.f, 0.f);
        for (int c = lo + tl; c < hi; c += ts) m = add2(m, each(lo, c));
        for (int o = ts / 2; o > 0; o >>= 1) m = add2(m, shfl_xor2(m, o));
        if (tl == 0 && lo < hi) give(k, lo, hi, m);
    }
}

// E values, or the codes of E values, from shared memory (addresses in the
// shared window: the loops over rows step 32-bit numbers).
template <typename T, int E> __device__ __forceinline__ Vals<T, E> held_chunk(uint32_t at) {
    Vals<T, E> c;
    constexpr int B = Vals<T, E>::B;
    if constexpr (B == 16)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(c.u[0]), "=r"(c.u[1]), "=r"(c.u[2]), "=r"(c.u[3]) : "r"(at));
    else if constexpr (B == 8)
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(c.u[0]), "=r"(c.u[1]) : "r"(at));
    else if constexpr (B == 4)
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(c.u[0]) : "r"(at));
    else
        asm volatile("ld.shared.u16 %0, [%1];" : "=r"(c.u[0]) : "r"(at));
    return c;
}
template <typename T, int E> __device__ __forceinline__ void held_values(uint32_t at, float (&v)[E]) { held_chunk<T, E>(at).get(v); }
__device__ __forceinline__ uint32_t held_byte(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}
template <int E> __device__ __forceinline__ void held_codes(uint32_t at, uint32_t b, float (&v)[E]) {
    if constexpr (E == 1) {
        v[0] = decode8((int8_t)held_byte(at)) * from_codes8(b);
    } else {
        const float f = from_codes8(b);
        float ff[E];
        fill_v(f, ff);
        uint32_t w[E / 4];
        if constexpr (E == 8)
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
        else
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at));
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            float q[4];
            decode8x4(w[i], q);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[4 * i + k] = q[k];
        }
        mul_v(v, ff, v);
    }
}

// The statistics' sums of the rows at `from` (shared window), n of them `step`
// bytes apart: K from the first of a thread's first call (n0 0).
template <typename T, int E>
__device__ __forceinline__ void sum_rows(uint32_t from, int n, uint32_t step, int n0, float (&minus_K)[E], float (&s1)[E], float (&s2)[E]) {
    if (n > 0 && n0 == 0) {
        held_values<T, E>(from, minus_K);
#pragma unroll
        for (int i = 0; i < E; ++i) minus_K[i] = -minus_K[i];
        from += step;
        --n;
    }
    for (; n >= 4; n -= 4) {
        Vals<T, E> c[4];
#pragma unroll
        for (int q = 0; q < 4; ++q, from += step) c[q] = held_chunk<T, E>(from);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float v[E];
            c[q].get(v);
            gn_deviate(v, minus_K, s1, s2);
        }
    }
    for (; n > 0; --n, from += step) {
        float v[E];
        held_values<T, E>(from, v);
        gn_deviate(v, minus_K, s1, s2);
    }
}

#define GN_DECLARE(suf)                                                          \
    const void *gn_flow_##suf(bool backward, int chunk, int act, bool kept);     \
    const void *gn_held_##suf(bool backward, int chunk, int act, bool kept);
GN_DECLARE(f32)
GN_DECLARE(bf16)
GN_DECLARE(f16)
#undef GN_DECLARE

}  // namespace rmsn
