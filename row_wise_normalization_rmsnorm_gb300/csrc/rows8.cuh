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
// The code of v f: adding 1.5 2^23 rounds to a whole number, ties to even,
// in the low bits (|v f| <= 128).
__device__ __forceinline__ int code8(float v, float f) {
    const float s = fminf(fmaxf(__fmul_rn(v, f), -127.f), 127.f);
    return (int)(__float_as_uint(__fadd_rn(s, 12582912.f)) & 0xffu);
}
__device__ __forceinline__ uint32_t codes8x4(float a, float b, float c, float d, float f) {
    return (uint32_t)code8(a, f) | (uint32_t)code8(b, f) << 8 | (uint32_t)code8(c, f) << 16 | (uint32_t)code8(d, f) << 24;
}
// Four codes as fp32: code + 128 as the low byte of 2^23, less 2^23 + 128.
__device__ __forceinline__ void decode8x4(uint32_t codes, float (&v)[4]) {
    const uint32_t u = codes ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + i)) - 8388736.f;
}
__device__ __forceinline__ float decode8(int8_t c) { return (float)c; }

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The codes of a chunk of E values and its block's scale. 32 / E neighbouring
// lanes hold a block and call this together; one whose chunk lies behind the
// row's end (`here` false, its values 0) writes nothing.
template <typename T, int E>
__device__ __forceinline__ void keep_chunk(const float (&v)[E], bool here, uint8_t *codes, uint8_t *scale) {
    constexpr int L = kBlock8 / E;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) top = max(top, abs_bits(v[i]));
    const uint32_t lane = threadIdx.x & 31u, mates = ((1u << L) - 1u) << (lane & ~(uint32_t)(L - 1));
#pragma unroll
    for (int o = 1; o < L; o <<= 1) top = max(top, __shfl_xor_sync(mates, top, o));
    const uint32_t b = scale8<T>(top);
    const float f = to_codes8(b);
    if (!here) return;
    if constexpr (E == 8)
        *reinterpret_cast<uint2 *>(codes) = make_uint2(codes8x4(v[0], v[1], v[2], v[3], f), codes8x4(v[4], v[5], v[6], v[7], f));
    else
        *reinterpret_cast<uint32_t *>(codes) = codes8x4(v[0], v[1], v[2], v[3], f);
    if ((lane & (L - 1)) == 0) *scale = (uint8_t)b;
}

}  // namespace rmsn
