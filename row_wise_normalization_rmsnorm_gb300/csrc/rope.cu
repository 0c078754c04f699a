// rope.cu -- rope_fwd, rope_bwd and paged_kv_append: rotary positions on
// head rows, and the same with a per-head RMSNorm before and a paged cache
// behind.
//
// The mathematics: frequency i of token t turns one pair of a head's values
// by the angle p f (position times frequency). The angle is reduced to a
// fraction of a turn in 64-bit integers (turn_by), since fp32's p f has
// lost its fraction where p is large, and the device's fp64 rate is too low
// to spend on it; sincospif takes the fraction.
//
// What bounds it: memory. Every value is read once and written once, at a
// few fp32 operations a value; the angles are shared by all heads of a
// token. So a warp takes one token and walks its heads, a group of lanes a
// head, the next heads' chunks on their way into shared memory by asynchronous
// copies (each lane reads back what it asked for: no barrier). The warp
// computes each angle once (two a lane for 64 frequencies) and hands them round
// in shared memory. With few tokens the heads are split over more warps.
// Measured (of 6770 GB/s, the copy rate): 16384 tokens of 40 heads by 128, bf16,
// 52.9 us, 94%; the append of 8192 tokens of 48 heads with their norm 39.2 us,
// 76%; the gradient of 4096 tokens, fp16, 18.4 us, 68%. The last two are few
// rounds of CTAs (2048 on 760 places, 1024 on 912): the gradient's second round
// has 112 CTAs and takes as long as one of 912.
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "head_rows.h"

namespace rmsn {

struct HeadSeg {
    const char *in;
    char *out;
    int64_t in_token, in_head;    // bytes
    int64_t out_token, out_head;  // bytes; a cache segment: page, head
    int64_t out_slot;             // bytes; cache segments only
    int heads;
};

struct RopeParams {
    HeadSeg seg[3];  // q, k, v
    const void *positions;
    const float *inv_freq;
    const int64_t *slots;
    const void *w[2];       // q's and k's norm weight, or NULL
    int64_t axis_stride;    // positions, in elements
    int64_t tokens, slots_end;
    uint32_t axis[8];       // two bits a frequency
    int naxes, pos64, half_dim, head_dim, adjacent;
    int page_size;
    int blocks, block_heads;  // head blocks a token, heads a block
    int items, lanes_log2;    // vector kernel: chunk pairs a head, lanes a head
    float sign;               // -1: the gradient's rotation
    float eps, offset, inv_n;
    int w32;
};

// (Plain loads throughout: the kernel may have been launched while the one
// before it was still writing what is read here after pdl_wait, which the
// non-coherent path does not provide for. With them the append of 8192 tokens
// takes 39.3 us instead of 37.6, the rotation of 16384 52.9 instead of 53.8.)

// ------------------------------------------------------------- angles --
// The angle p f is wanted modulo a turn, and fp32's p f has lost that where p
// is large. So the frequency is taken as a 64-bit fixed-point fraction of a
// turn, g = f / (2 pi) 2^64 (turn_step), and p g in wrapping integer
// arithmetic is the angle modulo a turn at once, exact but for g's last bit
// times p: below 2^-32 of a turn for |p| < 2^31 and |f| < 2. Of its top 32 bits
// fp32 holds 24: they are sincospif's argument, and the rest, an angle d below
// 2^-23, turns the result on by c - s d, s + c d. (Without d cos and sin were off
// by up to 1.9 units of 2^-24, with it by 1.4; the times are the same.)
__device__ __forceinline__ int64_t turn_step(float f) {
    constexpr uint64_t kPerTurn = 0xa2f9836e4e44152aull;  // 2^66 / (2 pi)
    const uint32_t bits = __float_as_uint(f) & 0x7fffffffu;
    const int ex = (int)(bits >> 23);
    // |f| = m 2^(ex - 150), m of 24 bits (a denormal's step is below one unit)
    const uint64_t m = (bits & 0x7fffffu) | 0x800000u;
    const uint64_t top = __umul64hi(m << 40, kPerTurn);  // m kPerTurn / 2^24
    const int shift = ex - 128;                          // g = top 2^(ex - 150 - 2 + 24)
    const uint64_t g = shift <= -64 ? 0 : (shift < 0 ? top >> -shift : (shift < 64 ? top << shift : 0));
    return f < 0.f ? -(int64_t)g : (int64_t)g;
}
__device__ __forceinline__ void turn_by(int64_t pos, int64_t step, float *c, float *s) {
    const int32_t a = (int32_t)(uint32_t)(((uint64_t)pos * (uint64_t)step) >> 32);  // 2^-31 of half a turn
    const float high = (float)a;
    // (high may be 2^31, which the conversion back holds to 2^31 - 1)
    const float d = (float)(a - __float2int_rn(high)) * (float)(3.14159265358979323846 * 0x1p-31);
    float c0, s0;
    sincospif(high * 0x1p-31f, &s0, &c0);
    *c = __fmaf_rn(-s0, d, c0);
    *s = __fmaf_rn(c0, d, s0);
}

__device__ __forceinline__ int64_t position(const RopeParams &p, int axis, int64_t t) {
    const int64_t i = (int64_t)axis * p.axis_stride + t;
    return p.pos64 ? static_cast<const int64_t *>(p.positions)[i]
                   : (int64_t) static_cast<const int32_t *>(p.positions)[i];
}

__device__ __forceinline__ int axis_of(const RopeParams &p, int i) { return (p.axis[i >> 4] >> (2 * (i & 15))) & 3; }

// cos and sin of the NF frequencies from i0 of token t.
template <int NF>
__device__ __forceinline__ void angles_of(const RopeParams &p, int64_t t, int i0, float *c, float *s) {
    int64_t at[ROPE_MAX_AXES];
    at[0] = position(p, 0, t);
#pragma unroll
    for (int a = 1; a < ROPE_MAX_AXES; ++a) at[a] = a < p.naxes ? position(p, a, t) : at[0];
#pragma unroll
    for (int i = 0; i < NF; ++i) {
        int64_t pos = at[0];
        if (p.naxes > 1) {
            const int a = axis_of(p, i0 + i);
            pos = a == 0 ? at[0] : a == 1 ? at[1] : a == 2 ? at[2] : at[3];
        }
        const float f = p.inv_freq[i0 + i];
        turn_by(pos, turn_step(f), c + i, s + i);
        if (!isfinite(f)) c[i] = s[i] = NAN;
        s[i] *= p.sign;
    }
}

// Where token t's row of head h (counted within its segment) is written;
// NULL: a token without a slot.
template <bool APPEND>
__device__ __forceinline__ char *row_out(const RopeParams &p, const HeadSeg &g, bool cache, int64_t t, int h,
                                         int64_t page, int place) {
    if (APPEND && cache) {
        if (page < 0) return nullptr;
        return g.out + page * g.out_token + place * g.out_slot + h * g.out_head;
    }
    return g.out + t * g.out_token + h * g.out_head;
}

// The page and the place in it of token t's slot; page -1: none.
__device__ __forceinline__ void find_slot(const RopeParams &p, int64_t t, int64_t &page, int &place) {
    const int64_t slot = p.slots[t];
    page = -1;
    place = 0;
    if (slot < 0 || slot >= p.slots_end) return;
    if (slot <= 0x7fffffffLL) {
        const uint32_t q = (uint32_t)slot / (uint32_t)p.page_size;
        page = q;
        place = (int)((uint32_t)slot - q * (uint32_t)p.page_size);
    } else {
        page = slot / p.page_size;
        place = (int)(slot - page * p.page_size);
    }
}

// ------------------------------------------------------------- chunks --
// A lane's unit of a row: V values in 16 bytes, or in 8 where rows are not
// whole 16-byte chunks (a half of 36 values of 16 bits).
template <typename T, int V> struct Chunk {
    static constexpr int W = V * (int)sizeof(T) / 4;  // words
    uint32_t w[W];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void from_shared(const void *p) {
        if constexpr (W == 4) {
            const uint4 v = lds128(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(smem_u32(p)));
        }
    }
    __device__ __forceinline__ void to_global(void *p) const {
        if constexpr (W == 4)
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
    __device__ __forceinline__ void unpack(float2 (&f)[V / 2]) const {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            if constexpr (std::is_same<T, float>::value)
                f[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
            else if constexpr (std::is_same<T, __half>::value)
                f[i] = f16x2_to_f2(w[i]);
            else
                f[i] = bf16x2_to_f2(w[i]);
        }
    }
    __device__ __forceinline__ void pack(const float2 (&f)[V / 2]) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            if constexpr (std::is_same<T, float>::value) {
                w[2 * i] = __float_as_uint(f[i].x);
                w[2 * i + 1] = __float_as_uint(f[i].y);
            } else if constexpr (std::is_same<T, __half>::value) {
                w[i] = f2_to_f16x2(f[i]);
            } else {
                w[i] = f2_to_bf16x2(f[i]);
            }
        }
    }
};

// offset + weight of the V values from element e (once a token and segment).
template <typename T, int V>
__device__ __forceinline__ void norm_factors(const RopeParams &p, const void *w, int e, float2 (&f)[V / 2]) {
#pragma unroll
    for (int q = 0; q < V / 2; ++q) {
        if (std::is_same<T, float>::value || p.w32) {
            const float2 v = reinterpret_cast<const float2 *>(static_cast<const float *>(w) + e)[q];
            f[q] = make_float2(p.offset + v.x, p.offset + v.y);
        } else if constexpr (!std::is_same<T, float>::value) {
            const uint32_t u = reinterpret_cast<const uint32_t *>(static_cast<const T *>(w) + e)[q];
            const float2 v = std::is_same<T, __half>::value ? f16x2_to_f2(u) : bf16x2_to_f2(u);
            f[q] = make_float2(p.offset + v.x, p.offset + v.y);
        }
    }
}

// ------------------------------------------------------ vectorised rows --
// A lane's two chunks of a head: the two halves of V pairs (half pairing),
// two neighbouring chunks of V / 2 pairs each (adjacent pairing), or two
// chunks of the values that pass unturned.
constexpr int kRopeThreads = 128;
constexpr int kRopeWarps = kRopeThreads / 32;
// Heads of a batch, batches under way, and the CTAs an SM that the registers
// are held to, without and with the norm. Measured together (bf16, 16384 tokens
// of 40 heads by 128, and the append of 8192 tokens of 48 with its norm; before
// the loads became plain ones): 53.6 and 37.4 us; one batch of three heads in
// registers instead 58.5 and 40.3; four batches 55.7 and 38.9; six CTAs for the
// norm too spill, 43.4. (Few tokens lost: the gradient of 4096 15.3 -> 16.6 us,
// calls one after the other.)
constexpr int kRopeUnroll = 2;
constexpr int kRopeDepth = 3;
constexpr int kRopeCtas[2] = {6, 5};

template <int BYTES> __device__ __forceinline__ void cp_async_chunk(void *dst, const void *src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the thread's newest N groups of copies have landed.
template <int N> __device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// FULL: every lane has two chunks of every head (head_dim = 2 V lanes a head,
// e.g. 64, 128 or 256 values of 16 bits), so nothing is tested a chunk.
template <typename T, int V, bool APPEND, bool NORM, bool ADJ, bool FULL>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas[NORM]) rope_vector(const __grid_constant__ RopeParams p) {
    constexpr int NP = V / 2, U = kRopeUnroll, CB = V * (int)sizeof(T);
    using PR = Pair<true>;
    __shared__ __align__(16) float2 turn[kRopeWarps][HEAD_MAX_DIM / 2];  // (cos, sin) of the warp's token
    constexpr int kDepth = kRopeDepth;
    __shared__ __align__(16) uint8_t places[kRopeWarps][kRopeDepth * kRopeUnroll * 64 * CB];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t unit = (int64_t)blockIdx.x * kRopeWarps + warp;
    pdl_wait();
    pdl_trigger();
    if (unit >= p.tokens * p.blocks) return;
    const int64_t t = unit / p.blocks;
    const int h0 = (int)(unit - t * p.blocks) * p.block_heads, h1 = h0 + p.block_heads;
    const int item = lane & ((1 << p.lanes_log2) - 1), grp = lane >> p.lanes_log2;
    const int step = 32 >> p.lanes_log2;
    const int rot_items = p.half_dim / V;
    const bool turns = item < rot_items;

    int e0, e1;
    if (turns) {
        e0 = ADJ ? item * 2 * V : item * V;
        e1 = ADJ ? e0 + V : e0 + p.half_dim;
    } else {
        e0 = 2 * p.half_dim + (item - rot_items) * 2 * V;
        e1 = e0 + V;
    }
    const bool has0 = FULL || e0 < p.head_dim, has1 = FULL || e1 < p.head_dim;
    const int b0 = e0 * (int)sizeof(T), b1 = e1 * (int)sizeof(T);

    // The heads of this block, segment by segment, in batches of U a group of
    // lanes. A lane's chunks of the next kDepth batches are on their way into
    // its own places in shared memory (copies that hold no registers), across
    // the segments' ends.
    constexpr int kSegs = APPEND ? 3 : 2;
    int hb[kSegs], he[kSegs];
    {
        int first = 0;
#pragma unroll
        for (int sg = 0; sg < kSegs; ++sg) {
            hb[sg] = max(h0 - first, 0);
            he[sg] = min(h1 - first, p.seg[sg].heads);
            first += p.seg[sg].heads;
        }
    }
    uint8_t *mine = places[warp] + lane * CB;  // [kDepth][U][2], 32 chunks apart
    int nsg = 0, nh = hb[0], slot = 0;  // the next batch to ask for; the next place
    auto ask = [&](int at) {
#pragma unroll
        for (int sg = 0; sg < kSegs; ++sg) {
            if (nsg != sg) continue;
            if (nh >= he[sg]) {  // (an empty segment too)
                ++nsg;
                if (sg + 1 < kSegs) nh = hb[sg + 1];
                continue;
            }
            const HeadSeg &g = p.seg[sg];
            const char *in = g.in + t * g.in_token;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = nh + u * step + grp;
                if (h < he[sg]) {
                    const char *row = in + h * g.in_head;
                    uint8_t *to = mine + (at * U + u) * 64 * CB;
                    if (has0) cp_async_chunk<CB>(to, row + b0);
                    if (has1) cp_async_chunk<CB>(to + 32 * CB, row + b1);
                }
            }
            nh += U * step;
            break;
        }
        cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kDepth; ++k) ask(k);

    int64_t page = 0;
    int place = 0;
    if (APPEND) find_slot(p, t, page, place);
    if (h0 < p.seg[0].heads + p.seg[1].heads) {
        for (int i = lane; i < p.half_dim; i += 32) {
            float c, s;
            angles_of<1>(p, t, i, &c, &s);
            turn[warp][i] = make_float2(c, s);
        }
        __syncwarp();
    }

#pragma unroll
    for (int sg = 0; sg < kSegs; ++sg) {
        if (hb[sg] >= he[sg]) continue;
        const HeadSeg &g = p.seg[sg];
        const bool cached = APPEND && sg > 0;
        char *out = cached ? g.out + page * g.out_token + place * g.out_slot : g.out + t * g.out_token;
        const bool kept = !cached || page >= 0;

        if (APPEND && sg == 2) {  // v: copied
#pragma unroll 1
            for (int h = hb[sg]; h < he[sg]; h += U * step) {
                cp_async_wait<kDepth - 1>();
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int hh = h + u * step + grp;
                    if (hh < he[sg] && kept) {
                        const uint8_t *from = mine + (slot * U + u) * 64 * CB;
                        char *row = out + hh * g.out_head;
                        Chunk<T, V> c;
                        if (has0) {
                            c.from_shared(from);
                            c.to_global(row + b0);
                        }
                        if (has1) {
                            c.from_shared(from + 32 * CB);
                            c.to_global(row + b1);
                        }
                    }
                }
                ask(slot);
                slot = slot + 1 == kDepth ? 0 : slot + 1;
            }
            continue;
        }

        // The turn's factors of this lane's pairs, the norm's weight folded
        // into them: y1 = x1 ca - x2 sb, y2 = x2 cb + x1 sa (times rstd).
        const void *w = NORM ? p.w[sg & 1] : nullptr;
        float2 ca[NP], sb[NP], cb[NP], sa[NP];
        {
            float2 fa[NP], fb[NP];
#pragma unroll
            for (int q = 0; q < NP; ++q) fa[q] = fb[q] = make_float2(1.f, 1.f);
            if (NORM && w) {
                if (has0) norm_factors<T, V>(p, w, e0, fa);
                if (has1) norm_factors<T, V>(p, w, e1, fb);
            }
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                ca[q] = fa[q];
                cb[q] = fb[q];
                sa[q] = sb[q] = make_float2(0.f, 0.f);
            }
            if (turns) {
#pragma unroll
                for (int q = 0; q < NP; ++q) {
                    // two frequencies of the lane's V
                    const float4 v = reinterpret_cast<const float4 *>(&turn[warp][item * V])[q];
                    if (!ADJ) {
                        const float2 c = make_float2(v.x, v.z), s = make_float2(v.y, v.w);
                        ca[q] = PR::mul(fa[q], c);
                        sb[q] = PR::mul(fb[q], make_float2(-s.x, -s.y));
                        cb[q] = PR::mul(fb[q], c);
                        sa[q] = PR::mul(fa[q], s);
                    } else {
                        // frequency i's pair (2i, 2i + 1) is one pair of registers, of
                        // the first chunk or the second; .x keeps the first value's
                        // factors, .y the second's
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int fi = 2 * q + h, at = fi % NP;
                            const float c = h ? v.z : v.x, s = h ? v.w : v.y;
                            const float2 ff = fi < NP ? fa[at] : fb[at];
                            const float2 cc = PR::mul(ff, make_float2(c, c)), ss = PR::mul(make_float2(ff.y, ff.x), make_float2(-s, s));
                            if (fi < NP) {
                                ca[at] = cc;
                                sa[at] = ss;
                            } else {
                                cb[at] = cc;
                                sb[at] = ss;
                            }
                        }
                    }
                }
            }
        }
        const bool raw = !turns && !(NORM && w);
#pragma unroll 1
        for (int h = hb[sg]; h < he[sg]; h += U * step) {
            cp_async_wait<kDepth - 1>();
            Chunk<T, V> x0[U], x1[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint8_t *from = mine + (slot * U + u) * 64 * CB;
                if (!FULL) {
                    x0[u].clear();
                    x1[u].clear();
                }
                if (has0) x0[u].from_shared(from);
                if (has1) x1[u].from_shared(from + 32 * CB);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int hh = h + u * step + grp;
                float2 a[NP], b[NP];
                x0[u].unpack(a);
                x1[u].unpack(b);
                float2 r2 = make_float2(1.f, 1.f);
                if (NORM && w) {  // (the same for the whole grid: the shuffles are uniform)
                    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                    for (int q = 0; q < NP; ++q) acc = PR::fma(a[q], a[q], PR::fma(b[q], b[q], acc));
                    float ss = acc.x + acc.y;
                    for (int o = (1 << p.lanes_log2) >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float r = rsqrtf(__fmaf_rn(ss, p.inv_n, p.eps));
                    r2 = make_float2(r, r);
                }
                if (hh >= he[sg] || !kept) continue;
#pragma unroll
                for (int q = 0; q < NP; ++q) {
                    float2 y0, y1;
                    if (!turns) {
                        y0 = PR::mul(a[q], ca[q]);
                        y1 = PR::mul(b[q], cb[q]);
                    } else if (!ADJ) {
                        y0 = PR::fma(b[q], sb[q], PR::mul(a[q], ca[q]));
                        y1 = PR::fma(a[q], sa[q], PR::mul(b[q], cb[q]));
                    } else {
                        y0 = PR::fma(make_float2(a[q].y, a[q].x), sa[q], PR::mul(a[q], ca[q]));
                        y1 = PR::fma(make_float2(b[q].y, b[q].x), sb[q], PR::mul(b[q], cb[q]));
                    }
                    a[q] = NORM ? PR::mul(y0, r2) : y0;
                    b[q] = NORM ? PR::mul(y1, r2) : y1;
                }
                char *row = out + hh * g.out_head;
                // (values that pass as they are keep their bits, a NaN's payload too)
                if (!raw) {
                    x0[u].pack(a);
                    x1[u].pack(b);
                }
                if (has0) x0[u].to_global(row + b0);
                if (has1) x1[u].to_global(row + b1);
            }
            // (the values read above have been used, so their places are free)
            ask(slot);
            slot = slot + 1 == kDepth ? 0 : slot + 1;
        }
    }
}

// --------------------------------------------------------- element-wise --
// Any head size, stride and alignment: a warp takes up to eight heads of a
// token, a lane one pair at a time; a head's sum of squares is taken in a
// pass of its own.
constexpr int kElemHeads = 8;

template <typename T, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads) rope_elements(const __grid_constant__ RopeParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    if (unit >= p.tokens * p.blocks) return;
    const int64_t t = unit / p.blocks;
    const int h0 = (int)(unit - t * p.blocks) * p.block_heads;
    const int hq = p.seg[0].heads, hqk = hq + p.seg[1].heads;
    const int htot = hqk + (APPEND ? p.seg[2].heads : 0);
    const int n = min(p.block_heads, htot - h0);
    int64_t page = 0;
    int place = 0;
    if (APPEND) find_slot(p, t, page, place);

    const T *in[kElemHeads];
    T *out[kElemHeads];
    float rstd[kElemHeads];
#pragma unroll
    for (int u = 0; u < kElemHeads; ++u) {
        in[u] = nullptr;
        out[u] = nullptr;
        rstd[u] = 1.f;
        if (u >= n) continue;
        const int h = h0 + u, sg = h < hq ? 0 : (h < hqk ? 1 : 2);
        const HeadSeg &g = p.seg[sg];
        const int hh = h - (sg == 0 ? 0 : sg == 1 ? hq : hqk);
        in[u] = reinterpret_cast<const T *>(g.in + t * g.in_token + hh * g.in_head);
        out[u] = reinterpret_cast<T *>(row_out<APPEND>(p, g, sg > 0, t, hh, page, place));
        if (APPEND && sg < 2 && p.w[sg]) {
            float ss = 0.f;
            for (int i = lane; i < p.head_dim; i += 32) {
                const float v = load_elem(in[u], i);
                ss = __fmaf_rn(v, v, ss);
            }
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            rstd[u] = rsqrtf(__fmaf_rn(ss, p.inv_n, p.eps));
        }
    }
    // value i of head u, normalised
    auto value = [&](int u, int sg, int i) {
        float v = load_elem(in[u], i);
        if (APPEND && sg < 2 && p.w[sg]) {
            const float w = std::is_same<T, float>::value || p.w32
                                ? load_elem(reinterpret_cast<const float *>(p.w[sg]), i)
                                : load_elem(reinterpret_cast<const T *>(p.w[sg]), i);
            v = v * rstd[u] * (p.offset + w);
        }
        return v;
    };
    for (int i = lane; i < p.half_dim; i += 32) {
        const int e0 = p.adjacent ? 2 * i : i, e1 = p.adjacent ? 2 * i + 1 : i + p.half_dim;
        float c = 1.f, s = 0.f;
        if (h0 < hqk) angles_of<1>(p, t, i, &c, &s);
#pragma unroll
        for (int u = 0; u < kElemHeads; ++u) {
            if (u >= n || !out[u]) continue;
            const int h = h0 + u, sg = h < hq ? 0 : (h < hqk ? 1 : 2);
            if (sg == 2) {  // v: copied
                out[u][e0] = in[u][e0];
                out[u][e1] = in[u][e1];
                continue;
            }
            const float a = value(u, sg, e0), b = value(u, sg, e1);
            store_elem(out[u], e0, __fmaf_rn(-b, s, a * c));
            store_elem(out[u], e1, __fmaf_rn(a, s, b * c));
        }
    }
    for (int i = 2 * p.half_dim + lane; i < p.head_dim; i += 32) {
#pragma unroll
        for (int u = 0; u < kElemHeads; ++u) {
            if (u >= n || !out[u]) continue;
            const int h = h0 + u, sg = h < hq ? 0 : (h < hqk ? 1 : 2);
            // (what passes as it is keeps its bits, a NaN's payload too)
            if (APPEND && sg < 2 && p.w[sg])
                store_elem(out[u], i, value(u, sg, i));
            else
                out[u][i] = in[u][i];
        }
    }
}

// ------------------------------------------------------------------ host --

static int elem_bytes(int dt) { return (dt & 0xff) == RMSNORM_F32 ? 4 : 2; }

template <typename T, int V, bool APPEND, bool NORM>
static int launch_vector(const RopeParams &p, const cudaLaunchConfig_t *cfg) {
    if constexpr (V * sizeof(T) == 16) {
        if (p.head_dim == 2 * V << p.lanes_log2)
            return p.adjacent ? (int)cudaLaunchKernelEx(cfg, rope_vector<T, V, APPEND, NORM, true, true>, p)
                              : (int)cudaLaunchKernelEx(cfg, rope_vector<T, V, APPEND, NORM, false, true>, p);
    }
    return p.adjacent ? (int)cudaLaunchKernelEx(cfg, rope_vector<T, V, APPEND, NORM, true, false>, p)
                      : (int)cudaLaunchKernelEx(cfg, rope_vector<T, V, APPEND, NORM, false, false>, p);
}

// vec: bytes of a chunk, 16 or 8; 0: element-wise.
template <typename T, bool APPEND>
static int launch_rope(int vec, const RopeParams &p, unsigned grid, cudaStream_t stream) {
    constexpr int V = 16 / (int)sizeof(T);
    LaunchCfg lc(grid, kRopeThreads, 0, stream);
    if (vec == 0) return (int)cudaLaunchKernelEx(&lc.cfg, rope_elements<T, APPEND>, p);
    if constexpr (APPEND) {
        if (p.w[0] || p.w[1])
            return vec == 16 ? launch_vector<T, V, true, true>(p, &lc.cfg) : launch_vector<T, V / 2, true, true>(p, &lc.cfg);
    }
    return vec == 16 ? launch_vector<T, V, APPEND, false>(p, &lc.cfg) : launch_vector<T, V / 2, APPEND, false>(p, &lc.cfg);
}

template <bool APPEND>
static int launch_rope_dt(int base, int vec, const RopeParams &p, unsigned grid, cudaStream_t s) {
    switch (base) {
    case RMSNORM_F32: return launch_rope<float, APPEND>(vec, p, grid, s);
    case RMSNORM_BF16: return launch_rope<__nv_bfloat16, APPEND>(vec, p, grid, s);
    default: return launch_rope<__half, APPEND>(vec, p, grid, s);
    }
}

// The angles' part of the parameters; false: an invalid argument.
static bool take_angles(const rope_angles_t &a, const uint8_t *axes, int head_dim, RopeParams &p) {
    if (!a.inv_freq || !on(a.inv_freq, 4)) return false;
    if (a.position_bytes != 4 && a.position_bytes != 8) return false;
    if (!on(a.positions, (uintptr_t)a.position_bytes)) return false;
    if (a.n_axes < 1 || a.n_axes > ROPE_MAX_AXES) return false;
    if (a.rotary_dim < 2 || a.rotary_dim % 2 != 0 || a.rotary_dim > head_dim) return false;
    if (a.pairing != ROPE_HALF && a.pairing != ROPE_ADJACENT) return false;
    p.positions = a.positions;
    p.inv_freq = a.inv_freq;
    p.axis_stride = a.n_axes > 1 ? a.axis_stride : 0;
    p.pos64 = a.position_bytes == 8;
    p.naxes = a.n_axes;
    p.half_dim = a.rotary_dim / 2;
    p.adjacent = a.pairing == ROPE_ADJACENT;
    for (int i = 0; axes && i < p.half_dim; ++i) {
        if (axes[i] >= a.n_axes) return false;
        p.axis[i >> 4] |= (uint32_t)axes[i] << (2 * (i & 15));
    }
    return true;
}

static HeadSeg segment(const rope_rows_t &r, int heads, int64_t tokens, int es) {
    HeadSeg g;
    std::memset(&g, 0, sizeof g);
    g.in = static_cast<const char *>(r.in);
    g.out = static_cast<char *>(r.out);
    g.in_token = stride_of(r.in_token, tokens) * es;
    g.in_head = stride_of(r.in_head, heads) * es;
    g.out_token = stride_of(r.out_token, tokens) * es;
    g.out_head = stride_of(r.out_head, heads) * es;
    g.heads = heads;
    return g;
}

static bool rows_apart(const rope_rows_t &r, int heads, int64_t tokens) {
    return heads == 0 || (apart(r.out_token, tokens) && apart(r.out_head, heads));
}
static bool seg_on(const HeadSeg &g, uintptr_t a) { return g.heads == 0 || (on(g.in, a) && on(g.out, a)); }
static bool seg_vec(const HeadSeg &g, int vec) {
    return g.heads == 0 || (on(g.in, vec) && on(g.out, vec) && g.in_token % vec == 0 && g.in_head % vec == 0 &&
                            g.out_token % vec == 0 && g.out_head % vec == 0 && g.out_slot % vec == 0);
}

// Geometry and launch, the segments and the rest of `p` being set.
template <bool APPEND>
static rmsnorm_status_t run_rope(RopeParams &p, int base, cudaStream_t stream) {
    const int es = elem_bytes(base);
    int sms = 0;
    int e = current_device(&sms, nullptr);
    if (e != 0) return head_cuda_fail(e);
    // the widest chunks that every array, stride and the two halves are made of
    // and that a warp's lanes hold a head in
    int vec = 16;
    for (; vec >= 8; vec /= 2) {
        const int V = vec / es;
        bool ok = p.half_dim % V == 0 && p.head_dim % V == 0;
        for (const HeadSeg &g : p.seg) ok = ok && seg_vec(g, vec);
        for (const void *w : p.w) ok = ok && on(w, p.w32 || es == 4 ? 8 : 4);
        p.items = p.half_dim / V + ((p.head_dim - 2 * p.half_dim) / V + 1) / 2;
        if (ok && p.items <= 32) break;
    }
    if (vec < 8) vec = 0;
    const int heads = p.seg[0].heads + p.seg[1].heads + p.seg[2].heads;
    if (vec) {
        while ((1 << p.lanes_log2) < p.items) ++p.lanes_log2;
        // One warp takes all heads of a token, so that their angles are
        // computed once, as long as that leaves eight warps an SM; with
        // fewer tokens the heads are halved until it does, down to one
        // round of the warp's lanes.
        const int round = 32 >> p.lanes_log2;
        p.block_heads = (heads + round - 1) / round * round;
        while (p.block_heads > round &&
               p.tokens * ((heads + p.block_heads - 1) / p.block_heads) < (int64_t)8 * sms)
            p.block_heads = (p.block_heads / round + 1) / 2 * round;
    } else {
        p.block_heads = kElemHeads;
        while (p.block_heads > 1 && p.tokens * ((heads + p.block_heads - 1) / p.block_heads) < (int64_t)8 * sms)
            p.block_heads /= 2;
    }
    p.blocks = (heads + p.block_heads - 1) / p.block_heads;
    const int64_t warps = p.tokens * p.blocks;
    const int64_t grid = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    if (grid > 0x7fffffffLL) return RMSNORM_ERR_UNSUPPORTED;
    e = launch_rope_dt<APPEND>(base, vec, p, (unsigned)grid, stream);
    return e == 0 ? RMSNORM_SUCCESS : head_cuda_fail(e);
}

static rmsnorm_status_t rope_impl(const rope_call_t *c, const uint8_t *axes, float sign, cudaStream_t stream) {
    if (!c) return RMSNORM_ERR_INVALID_ARG;
    if (c->dtype != RMSNORM_F32 && c->dtype != RMSNORM_BF16 && c->dtype != RMSNORM_F16) return RMSNORM_ERR_INVALID_ARG;
    if (c->head_dim < 1 || c->head_dim > HEAD_MAX_DIM || c->tokens < 0 || c->tokens > 0x7fffffffLL ||
        c->q_heads < 1 || c->k_heads < 0 || c->q_heads > 65535 || c->k_heads > 65535)
        return RMSNORM_ERR_INVALID_ARG;
    RopeParams p;
    std::memset(&p, 0, sizeof p);
    if (!take_angles(c->angles, axes, c->head_dim, p)) return RMSNORM_ERR_INVALID_ARG;
    if (c->tokens == 0) return RMSNORM_SUCCESS;
    const int es = elem_bytes(c->dtype);
    if (!c->angles.positions || !c->q.in || !c->q.out || (c->k_heads && (!c->k.in || !c->k.out)))
        return RMSNORM_ERR_INVALID_ARG;
    if (!rows_apart(c->q, c->q_heads, c->tokens) || !rows_apart(c->k, c->k_heads, c->tokens)) return RMSNORM_ERR_INVALID_ARG;
    p.seg[0] = segment(c->q, c->q_heads, c->tokens, es);
    p.seg[1] = segment(c->k, c->k_heads, c->tokens, es);
    if (!seg_on(p.seg[0], es) || !seg_on(p.seg[1], es)) return RMSNORM_ERR_INVALID_ARG;
    p.tokens = c->tokens;
    p.head_dim = c->head_dim;
    p.sign = sign;
    return run_rope<false>(p, c->dtype, stream);
}

}  // namespace rmsn

using namespace rmsn;

extern "C" rmsnorm_status_t rope_fwd(const rope_call_t *call, const uint8_t *axes, rmsnorm_stream_t stream) {
    return rope_impl(call, axes, 1.f, (cudaStream_t)stream);
}

extern "C" rmsnorm_status_t rope_bwd(const rope_call_t *call, const uint8_t *axes, rmsnorm_stream_t stream) {
    return rope_impl(call, axes, -1.f, (cudaStream_t)stream);
}

extern "C" rmsnorm_status_t paged_kv_append(const paged_append_call_t *c, const uint8_t *axes,
                                            rmsnorm_stream_t stream) {
    if (!c) return RMSNORM_ERR_INVALID_ARG;
    const int base = c->dtype & ~RMSNORM_WEIGHT_F32;
    if (base != RMSNORM_F32 && base != RMSNORM_BF16 && base != RMSNORM_F16) return RMSNORM_ERR_INVALID_ARG;
    const paged_cache_t &pc = c->cache;
    if (c->head_dim < 1 || c->head_dim > HEAD_MAX_DIM || c->tokens < 0 || c->tokens > 0x7fffffffLL ||
        c->q_heads < 0 || c->q_heads > 65535 || pc.heads < 1 || pc.heads > 65535)
        return RMSNORM_ERR_INVALID_ARG;
    if (pc.page_size < 1 || pc.pages < 0 || pc.pages > INT64_MAX / pc.page_size) return RMSNORM_ERR_INVALID_ARG;
    if (!std::isfinite(c->eps) || !std::isfinite(c->offset) || c->eps < 0.f) return RMSNORM_ERR_INVALID_ARG;
    RopeParams p;
    std::memset(&p, 0, sizeof p);
    if (c->angles.positions && !take_angles(c->angles, axes, c->head_dim, p)) return RMSNORM_ERR_INVALID_ARG;
    if (c->tokens == 0) return RMSNORM_SUCCESS;
    const int es = elem_bytes(base);
    if (!c->k.in || !c->v.in || !c->slots || !on(c->slots, 8) || !pc.k || !pc.v ||
        (c->q_heads && (!c->q.in || !c->q.out)))
        return RMSNORM_ERR_INVALID_ARG;
    if (!rows_apart(c->q, c->q_heads, c->tokens) || !apart(pc.k_page, pc.pages) || !apart(pc.k_slot, pc.page_size) ||
        !apart(pc.k_head, pc.heads) || !apart(pc.v_page, pc.pages) || !apart(pc.v_slot, pc.page_size) ||
        !apart(pc.v_head, pc.heads))
        return RMSNORM_ERR_INVALID_ARG;
    const uintptr_t wes = (c->dtype & RMSNORM_WEIGHT_F32) ? 4 : (uintptr_t)es;
    if (!on(c->wq, wes) || !on(c->wk, wes)) return RMSNORM_ERR_INVALID_ARG;
    p.seg[0] = segment(c->q, c->q_heads, c->tokens, es);
    auto cached = [&](const rope_rows_t &r, void *cache, int64_t page, int64_t slot, int64_t head) {
        HeadSeg g = segment(r, pc.heads, c->tokens, es);
        g.out = static_cast<char *>(cache);
        g.out_token = stride_of(page, pc.pages) * es;
        g.out_slot = stride_of(slot, pc.page_size) * es;
        g.out_head = stride_of(head, pc.heads) * es;
        return g;
    };
    p.seg[1] = cached(c->k, pc.k, pc.k_page, pc.k_slot, pc.k_head);
    p.seg[2] = cached(c->v, pc.v, pc.v_page, pc.v_slot, pc.v_head);
    for (const HeadSeg &g : p.seg)
        if (!seg_on(g, es)) return RMSNORM_ERR_INVALID_ARG;
    p.slots = c->slots;
    p.slots_end = pc.pages * pc.page_size;
    p.page_size = pc.page_size;
    p.w[0] = c->q_heads ? c->wq : nullptr;
    p.w[1] = c->wk;
    p.w32 = (c->dtype & RMSNORM_WEIGHT_F32) ? 1 : 0;
    p.tokens = c->tokens;
    p.head_dim = c->head_dim;
    p.sign = 1.f;
    p.eps = c->eps;
    p.offset = c->offset;
    p.inv_n = 1.f / (float)c->head_dim;
    return run_rope<true>(p, base, (cudaStream_t)stream);
}
