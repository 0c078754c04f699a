// rows8.cuh -- rows held in 8 bits (activation checkpoints), as the kernels
// that write and read them see them.
//
// A row's values lie in blocks of 32 neighbours (the last one may be
// shorter). A block has one scale byte b, standing for 2^(b - 127), and a
// value is kept as the whole number nearest to value / 2^(b - 127), ties to
// even, -127 .. 127. b is the smallest that holds the block's largest
// magnitude a = m 2^e (1 <= m < 2): a / 2^(e - 6) = 64 m lies in [64, 128)
// and rounds to 127 at most where m < 255/128, else the scale doubles. So b
// comes from the bits of a alone: (bits(a) + 2^16) >> 23 carries into the
// exponent exactly where m >= 255/128, and multiplying by a power of two is
// exact: codes have no rounding but their own. An error is at most half a
// step, 2^-7 of the block's largest magnitude (1 / 127.5 where m = 255/128).
// The step stops at the largest whose 64 is still a finite value of the
// storage type (fp16 2^9, else 2^121): there a value may be one step off.
// A block with an infinity or a NaN gets b = 255 and stands for NaN.
#pragma once

#include "common.cuh"

namespace rmsn {

constexpr int kBlock8 = 32;          // values that share a scale
constexpr uint32_t kScaleNone = 255;  // a block that is not finite

template <typename T> struct MostScale { static constexpr uint32_t b = 127 + 121; };
template <> struct MostScale<__half> { static constexpr uint32_t b = 127 + 9; };

// The scale byte from the bits of the block's largest magnitude.
template <typename T> __device__ __forceinline__ uint32_t scale8(uint32_t abs_bits) {
    if (abs_bits >= 0x7f800000u) return kScaleNone;
    const int b = (int)((abs_bits + 0x10000u) >> 23) - 6;
    return (uint32_t)min(max(b, 0), (int)MostScale<T>::b);
}
// 2^(127 - b), what a value is multiplied by to be coded (0 for kScaleNone:
// whatever the codes are, the block stands for NaN).
__device__ __forceinline__ float to_codes8(uint32_t b) {
    return b == kScaleNone ? 0.f : __uint_as_float((254u - b) << 23);
}
// 2^(b - 127), what a code is multiplied by (2^-127 is a subnormal).
__device__ __forceinline__ float from_codes8(uint32_t b) {
    return b == kScaleNone ? __uint_as_float(0x7fc00000u) : b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}
// The code of v f, in the low byte: adding 1.5 2^23 rounds to a whole number,
// ties to even (one fma: the product is exact). |v f| < 127.5 but for a block
// at the largest scale, whose steps are held to 127.
__device__ __forceinline__ float held8(float steps) { return fminf(fmaxf(steps, -127.f), 127.f); }
__device__ __forceinline__ uint8_t code8(float v, uint32_t b) {
    return (uint8_t)__float_as_uint(__fadd_rn(held8(__fmul_rn(v, to_codes8(b))), 12582912.f));
}
// Four codes, lowest byte first.
__device__ __forceinline__ uint32_t codes8x4(float2 a, float2 b, float f) {
    const float2 ff = make_float2(f, f), magic = make_float2(12582912.f, 12582912.f);
    a = Pair<true>::fma(a, ff, magic);
    b = Pair<true>::fma(b, ff, magic);
    const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}
// Four codes as fp32: code + 128 as the low byte of 2^23, less 2^23 + 128.
__device__ __forceinline__ void decode8x4(uint32_t codes, float (&v)[4]) {
    const uint32_t u = codes ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + i)) - 8388736.f;
}
__device__ __forceinline__ float decode8(int8_t c) { return (float)c; }

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The bits of a chunk's largest magnitude (E values in w), combined over the
// 32 / E neighbouring lanes that hold its block. 16-bit types are compared as
// pairs of 16-bit numbers (magnitudes are in the order of their bits).
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <typename T, int E> __device__ __forceinline__ uint32_t block_top(const uint32_t *w, uint32_t lanes) {
    constexpr int L = kBlock8 / E, N = E * (int)sizeof(T) / 4;
    constexpr uint32_t mag = sizeof(T) == 2 ? 0x7fff7fffu : 0x7fffffffu;
    auto most = [](uint32_t a, uint32_t b) { return sizeof(T) == 2 ? max_u16x2(a, b) : max(a, b); };
    uint32_t m = w[0] & mag;
#pragma unroll
    for (int i = 1; i < N; ++i) m = most(m, w[i] & mag);
#pragma unroll
    for (int o = 1; o < L; o <<= 1) m = most(m, __shfl_xor_sync(lanes, m, o));
    if constexpr (sizeof(T) == 4) return m;
    m = max(m & 0xffffu, m >> 16);
    if constexpr (std::is_same<T, __half>::value) return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
    return m << 16;
}
// The lanes of this one's block.
template <int E> __device__ __forceinline__ uint32_t block_lanes() {
    constexpr int L = kBlock8 / E;
    return ((1u << L) - 1u) << ((threadIdx.x & 31u) & ~(uint32_t)(L - 1));
}

// The codes of a chunk of E values (8 or 4, in w) and its block's scale. The
// lanes of a block call this together; one whose chunk lies behind the row's
// end (`here` false, the chunk zeros) writes nothing. `lanes`: those of the
// block, or all 32 where the whole warp is here.
template <typename T, int E>
__device__ __forceinline__ void keep_chunk(const uint32_t *w, bool here, uint32_t lanes, uint8_t *codes, uint8_t *scale) {
    const uint32_t b = scale8<T>(block_top<T, E>(w, lanes));
    if (!here) return;
    float f = to_codes8(b);
    float2 v[E / 2];
#pragma unroll
    for (int q = 0; q < E / 2; ++q) {
        if constexpr (sizeof(T) == 4)
            v[q] = make_float2(__uint_as_float(w[2 * q]), __uint_as_float(w[2 * q + 1]));
        else if constexpr (std::is_same<T, __half>::value)
            v[q] = f16x2_to_f2(w[q]);
        else
            v[q] = bf16x2_to_f2(w[q]);
    }
    if (b == MostScale<T>::b) {
#pragma unroll
        for (int q = 0; q < E / 2; ++q) v[q] = make_float2(held8(v[q].x * f), held8(v[q].y * f));
        f = 1.f;
    }
    if constexpr (E == 8)
        *reinterpret_cast<uint2 *>(codes) = make_uint2(codes8x4(v[0], v[1], f), codes8x4(v[2], v[3], f));
    else
        *reinterpret_cast<uint32_t *>(codes) = codes8x4(v[0], v[1], f);
    if ((threadIdx.x & (kBlock8 / E - 1)) == 0) *scale = (uint8_t)b;
}
template <typename T>
__device__ __forceinline__ void keep_chunk(const uint4 &c, bool here, uint32_t lanes, uint8_t *codes, uint8_t *scale) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    keep_chunk<T, Elem<T>::E>(w, here, lanes, codes, scale);
}

}  // namespace rmsn
