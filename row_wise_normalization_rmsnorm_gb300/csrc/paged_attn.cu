// paged_attn.cu -- paged_attn_fwd: attention of new tokens over a paged
// key/value cache, on the tensor cores.
//
// The mathematics, per row (one query head of one new token), over the key
// tiles in order with running maximum m, sum l and accumulator o:
//   s = q K^T,  m' = max(m, max s),  p = 2^(c (s - m')),  c = scale log2 e
//   l = l 2^(c (m - m')) + sum p,    o = o 2^(c (m - m')) + p V
// and at the end o / l and (c m + log2 l) ln 2. The maximum that p is taken
// against only has to be near the true one: o and l are rescaled only when
// the true maximum has grown by more than 2^8, so p stays below 2^8 and the
// rescaling is rare (both ends of fp16 and fp32 are far away).
//
// Rows: the query heads that share a key head are rows of one tile (row =
// token * group + head in group), so a decoding step reads each key once
// for all of them.
//
// Two geometries (NQ tiles of 128 rows a CTA):
//  NQ = 2, prompts and chunks: 256 rows a CTA and one CTA an SM. Bound by
//    the matrix instructions; while the softmax of one tile runs, the other
//    tile's two products do.
//  NQ = 1, few rows (decoding): at most 64 rows, two CTAs an SM, the keys
//    split over CTAs where there are too few of them. Bound by the cache's
//    bytes; the two CTAs cover each other's latencies.
//
// Roles: four warps a tile for the softmax (a thread owns a row: no
// shuffles), one warp copying K and V tiles (one TMA box a page, or part of
// a page), one thread issuing matrix instructions. S and p share tensor
// memory (p, as the 16-bit A operand of the second product, overwrites s);
// o accumulates in tensor memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "head_rows.h"
#include "tcgen05.cuh"

namespace rmsn {

constexpr int kKeyTile = 128;
constexpr uint32_t kAttnWait = 1u << 22;         // polls of one barrier ...
constexpr uint64_t kAttnWaitNs = 2000000000ull;  // ... and time, before a kernel gives up
constexpr float kRescale = 8.f;           // log2 of how far a row's reference maximum may lag

struct AttnParams {
    const char *q;
    char *out;
    float *lse;
    float *part_o;    // [splits][T * heads][D] or NULL (one split)
    float *part_lse;  // [splits][T * heads], base 2
    const int32_t *table, *kv_lens, *cu_q;
    int64_t q_token, q_head, out_token, out_head;  // bytes
    int64_t table_stride;
    int64_t tokens;
    int *status;
    float c;  // scale * log2(e)
    int batch, width, heads, kv_heads, group, head_dim, pages, page_size, box_rows;
    int max_q, max_kv, causal, q_tiles, splits, chunk;  // chunk: keys a split takes
    int tile_toks;                                      // tokens a row tile takes
    int q_tma, q_vec, out_vec;
};

template <int DP, int NQ>
struct AttnShape {
    static constexpr int kHalves = DP / 64;
    static constexpr int kQRows = NQ == 2 ? 128 : 64;  // rows held of a tile
    static constexpr int kQBytes = kQRows * DP * 2;
    static constexpr int kStage = kKeyTile * DP * 2;
    static constexpr int kStages = NQ == 2 ? (DP == 128 ? 5 : 8) : (DP == 128 ? 3 : 6);
    static constexpr int kBars = NQ * kQBytes + kStages * kStage;
    static constexpr int kSmem = kBars + 256;
    // NQ == 2: the copy and issue warps fill up a warpgroup of their own, so
    // that registers can move to the softmax warps: 168 a thread at launch,
    // then 2 x 128 x 208 + 128 x 88 = 384 x 168
    static constexpr int kThreads = NQ == 2 ? 384 : 192;
    // tensor memory: s (and p) of each tile, then o of each tile
    static constexpr uint32_t kO = NQ * kKeyTile;
    static constexpr uint32_t kCols = NQ == 2 ? 512 : 256;
    static_assert(kO + NQ * DP <= kCols, "tensor memory");
    // an NQ == 1 tile's matrix instruction reads 128 rows where 64 are held:
    // the rest, other parts of this CTA's shared memory, only feeds rows
    // that nothing reads
    static_assert((kHalves - 1) * kQRows * 128 + 128 * 128 <= kBars, "q operand inside shared memory");
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

template <typename T> __device__ __forceinline__ uint32_t pack_pair(float2 v);
template <> __device__ __forceinline__ uint32_t pack_pair<__nv_bfloat16>(float2 v) { return f2_to_bf16x2(v); }
template <> __device__ __forceinline__ uint32_t pack_pair<__half>(float2 v) { return f2_to_f16x2(v); }

__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// A CTA's waits: bounded, and given up by all roles once one of them did.
struct Waiter {
    volatile int *gave_up;  // shared memory
    int *status;
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) const {
        if (mbar_try_wait_cta(bar, parity)) return true;
        const uint64_t began = now_ns();
        for (uint32_t i = 0; i < kAttnWait; ++i) {
            if (mbar_try_wait_cta(bar, parity)) return true;
            if ((i & 15u) == 15u && (*gave_up || now_ns() - began > kAttnWaitNs)) break;
        }
        *gave_up = 1;
        *status = 1;
        return false;
    }
};

template <typename T, int DP, int NQ>
__global__ void __launch_bounds__(NQ == 2 ? 384 : 192, NQ == 2 ? 1 : 2)
    paged_attn(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap qmap,
               const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using S = AttnShape<DP, NQ>;
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int NST = S::kStages;
    constexpr int kProducer = NQ * 4, kIssuer = NQ * 4 + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    pdl_wait();
    pdl_trigger();

    // ---- which rows and keys: (b, key head) fastest, then the split, then
    // the row tile, last rows (most keys) first
    int id = blockIdx.x;
    const int kvh = id % p.kv_heads;
    id /= p.kv_heads;
    const int b = id % p.batch;
    id /= p.batch;
    const int split = id % p.splits;
    const int qt = p.q_tiles - 1 - id / p.splits;
    const int T_ = (int)p.tokens;
    const int q0 = min(max(__ldg(p.cu_q + b), 0), T_);
    const int nq = min(max(__ldg(p.cu_q + b + 1), q0), T_) - q0;  // the sequence's new tokens
    const int nq_out = min(nq, p.max_q);                           // those that are written
    const int kv = max(0, min(min(__ldg(p.kv_lens + b), p.max_kv), (int)min((int64_t)p.width * p.page_size, (int64_t)0x7fffffff)));
    const int tt = p.tile_toks, tok0 = qt * NQ * tt;
    const int toks = min(nq_out - tok0, NQ * tt);  // the CTA's tokens, tt a tile
    if (toks <= 0) return;
    // keys that the CTA's last row sees, and this split's part of them
    const int last_tok = tok0 + toks - 1;
    const int64_t lim = p.causal ? min((int64_t)kv, max((int64_t)0, (int64_t)kv - nq + last_tok + 1)) : kv;
    const int64_t kbeg64 = (int64_t)split * p.chunk;
    const int64_t kend64 = p.splits > 1 ? min(lim, kbeg64 + p.chunk) : lim;
    if (p.splits > 1 && kend64 <= kbeg64) return;
    const int kbeg = (int)kbeg64, kend = (int)kend64;
    const int ntiles = (kend - kbeg + kKeyTile - 1) / kKeyTile;
    const int act = toks > tt ? 2 : 1;  // tiles with rows
    const int last_valid = kv - (kbeg + (ntiles - 1) * kKeyTile);  // cached keys of the last tile
    const bool fix = ntiles > 0 && last_valid < kKeyTile && last_valid % p.box_rows != 0;

    if ((smem_u32(smem) & 1023u) != 0) {  // the swizzle goes by the address
        if (threadIdx.x == 0) *p.status = 1;
        return;
    }
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::kBars);
    uint64_t *full = bars, *empty = bars + NST;
    uint64_t *s_ready = empty + NST, *p_half = s_ready + NQ, *p_ready = p_half + NQ, *o_done = p_ready + NQ;
    uint64_t *q_ready = o_done + NQ, *v_fixed = q_ready + 1, *drained = v_fixed + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drained + 1);
    volatile int *gave_up = reinterpret_cast<volatile int *>(tmem_slot + 1);
    static_assert((2 * S::kStages + 4 * NQ + 3) * 8 + 8 <= 256, "barriers");

    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int t = 0; t < NQ; ++t) {
            const int live = min(max(toks - t * tt, 0), tt) * p.group;  // rows of the tile
            mbar_init(s_ready + t, 1);
            mbar_init(p_half + t, live > 0 ? (live + 31) / 32 : 1);  // its warps with rows
            mbar_init(p_ready + t, live > 0 ? (live + 31) / 32 : 1);
            mbar_init(o_done + t, 1);
        }
        mbar_init(q_ready, p.q_tma ? 1 : NQ * 4);
        mbar_init(v_fixed, 1);
        mbar_init(drained, 1);
        *gave_up = 0;
        mbar_init_fence();
    }
    if (warp == kIssuer) tmem_alloc(tmem_slot, S::kCols);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = *tmem_slot;
    const Waiter wait{gave_up, p.status};
    // for a whole warp: all of it goes on or none
    auto warp_wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
    volatile int still = 0;  // the last waits, after giving up, have a limit of their own
    const uint32_t sbase = smem_u32(smem);
    const uint32_t stage0 = sbase + NQ * S::kQBytes;

    if (warp >= kProducer) {
    if constexpr (NQ == 2) fewer_registers<88>();
    if (warp == kProducer) {
        // ---------------------------------------------------- K and V copies
        // A tile is 128 / box_rows boxes by 64 columns; lane l copies piece
        // l % boxes of half l / boxes.
        const int boxes = kKeyTile / p.box_rows;
        const int piece = lane % boxes, half = lane / boxes;
        const bool copies = half < S::kHalves;
        const uint32_t off = (uint32_t)(half * kKeyTile * 128 + piece * p.box_rows * 128);
        auto find = [&](int tile, int &page, int &place) {
            const int key = kbeg + tile * kKeyTile + piece * p.box_rows;
            page = p.pages;  // outside the cache: zeros
            place = 0;
            if (copies && tile < ntiles && key < kv) {
                const int col = key / p.page_size;
                const int id = __ldg(p.table + b * p.table_stride + col);
                if (id >= 0 && id < p.pages) page = id;
                place = key - col * p.page_size;
            }
        };
        int page, place, next_page, next_place;
        find(0, page, place);
        if (p.q_tma && lane == 0) {
            // q's rows: tt tokens of `group` heads are one box, row after row
            mbar_arrive_expect_tx(q_ready, (uint32_t)(act * S::kHalves * tt * p.group * 128));
            for (int t = 0; t < act; ++t)
                for (int h = 0; h < S::kHalves; ++h)
                    tile_g2s(sbase + t * S::kQBytes + h * (S::kQRows * 128), &qmap, h * 64, 0, kvh, q0 + tok0 + t * tt, q_ready);
        }
        __syncwarp();
        int issued = 0;
        bool ok = true;
        for (int j = 0; j < ntiles && ok; ++j) {
            find(j + 1, next_page, next_place);
#pragma unroll
            for (int kvsel = 0; kvsel < 2; ++kvsel) {
                const int st = issued % NST;
                if (issued >= NST && !warp_wait(empty + st, (uint32_t)((issued / NST - 1) & 1))) {
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(full + st, S::kStage);
                __syncwarp();
                if (copies)
                    tile_g2s(stage0 + st * S::kStage + off, kvsel ? &vmap : &kmap, half * 64, place, kvh, page, full + st);
                ++issued;
            }
            page = next_page;
            place = next_place;
        }
        if (fix && ok) {
            // Values past the sequence's end in its last page would meet a
            // zero weight, and 0 * NaN is NaN: they become zeros.
            const int st = (issued - 1) % NST;
            if (warp_wait(full + st, (uint32_t)(((issued - 1) / NST) & 1))) {
                const int end = (last_valid / p.box_rows + 1) * p.box_rows;  // later boxes are zeros
                const int chunks = (end - last_valid) * 8;
                for (int i = lane; i < chunks * S::kHalves; i += 32) {
                    const int h = i / chunks, c = i - h * chunks;
                    sts128(smem + NQ * S::kQBytes + st * S::kStage + h * kKeyTile * 128 + last_valid * 128 + c * 16,
                           make_uint4(0, 0, 0, 0));
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(v_fixed);
            }
        }
        if (*gave_up) {  // no copy may be in flight when the CTA ends
            const Waiter last{&still, p.status};
            if (p.q_tma) last(q_ready, 0);
            for (int i = max(0, issued - NST); i < issued; ++i) last(full + i % NST, (uint32_t)((i / NST) & 1));
        }
    } else if (warp == kIssuer) {
        // ------------------------------------------- the matrix instructions
        // The whole warp walks the tiles (operands stay uniform), one lane issues.
        const bool issues = elect_one();
        const int ksteps = (p.head_dim + 15) / 16;
        const uint32_t qk_word = mma_word(std::is_same<T, __nv_bfloat16>::value, 128, kKeyTile, 0);
        const uint32_t pv_word = mma_word(std::is_same<T, __nv_bfloat16>::value, 128, (uint32_t)ksteps * 16, 1);
        const uint64_t q_op = smem_operand(sbase, 16, 1024);
        const uint64_t k_op = smem_operand(stage0, 16, 1024);
        const uint64_t v_op = smem_operand(stage0, kKeyTile * 128, 1024);
        // (an operand's address field counts 16 bytes)
        auto qk = [&](int t, int st) {
            if (issues) {
                const uint64_t a = q_op + (uint64_t)(t * S::kQBytes / 16), b = k_op + (uint64_t)(st * (S::kStage / 16));
#pragma unroll
                for (int i = 0; i < DP / 16; ++i) {
                    const int h = i >> 2, o = (i & 3) * 2;
                    if (i < ksteps)
                        mma_ss(tmem + t * kKeyTile, a + (uint64_t)(h * (S::kQRows * 8) + o), b + (uint64_t)(h * (kKeyTile * 8) + o),
                               qk_word, i > 0);
                }
                mma_commit(s_ready + t);
            }
            __syncwarp();
        };
        // half the keys' product
        auto pv = [&](int t, int st, int half, bool add) {
            if (issues) {
                const uint64_t b = v_op + (uint64_t)(st * (S::kStage / 16) + half * (kKeyTile / 32) * 128);
                const uint32_t a = tmem + t * kKeyTile + half * (kKeyTile / 4);
#pragma unroll
                for (int i = 0; i < kKeyTile / 32; ++i)
                    mma_ts(tmem + S::kO + t * DP, a + i * 8, b + (uint64_t)(i * 128), pv_word, add || i > 0);
                if (half) mma_commit(o_done + t);
            }
            __syncwarp();
        };
        auto free_stage = [&](int n) {
            if (issues) mma_commit(empty + n % NST);
            __syncwarp();
        };
        // stage and phase of the ring's n-th tile (K_0, V_0, K_1, V_1, ...)
        auto arrived = [&](int n) { return warp_wait(full + n % NST, (uint32_t)((n / NST) & 1)); };
        bool ok = warp_wait(q_ready, 0) && (ntiles == 0 || arrived(0));
        if (ok && ntiles > 0) {
            tc_after_sync();
            for (int t = 0; t < act; ++t) qk(t, 0);
            free_stage(0);
            ok = arrived(1);
        }
        for (int j = 0; j < ntiles && ok; ++j) {
            const bool more = j + 1 < ntiles;
            if (!more && fix) ok = warp_wait(v_fixed, 0);
            for (int t = 0; t < act && ok; ++t) {
                if (!(ok = warp_wait(p_half + t, (uint32_t)(j & 1)))) break;
                tc_after_sync();
                pv(t, (2 * j + 1) % NST, 0, j > 0);
                if (!(ok = warp_wait(p_ready + t, (uint32_t)(j & 1)))) break;
                tc_after_sync();
                pv(t, (2 * j + 1) % NST, 1, true);
                if (t == act - 1) free_stage(2 * j + 1);
                if (more) {
                    if (t == 0) ok = arrived(2 * j + 2);
                    if (ok) qk(t, (2 * j + 2) % NST);
                    // (here, where the products just issued cover the wait)
                    if (ok && t == 0) ok = arrived(2 * j + 3);
                }
            }
            if (more && ok) free_stage(2 * j + 2);
        }
        if (*gave_up) {  // nor may a matrix instruction be
            __syncwarp();
            if (issues) mma_commit(drained);
            Waiter{&still, p.status}(drained, 0);
        }
    }
    } else {
        // --------------------------------------------------------- softmax
        if constexpr (NQ == 2) more_registers<208>();
        const int t = warp >> 2, r = threadIdx.x & 127;  // tile, row in it
        if (!p.q_tma) {
            // q that a tiled copy does not take (bases or strides off 16-byte
            // boundaries): eight chunks in flight a thread, to the swizzled rows,
            // zeros past the rows and head_dim
            constexpr int kChunks = S::kHalves * 8, kBatch = 8;
            const int rows = min(max(toks - t * tt, 0), tt) * p.group, hd_chunks = p.head_dim / 8;
            for (int i0 = r; i0 < S::kQRows * kChunks; i0 += 128 * kBatch) {
                uint4 v[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int i = i0 + u * 128, rr = i / kChunks, c = i % kChunks;
                    v[u] = make_uint4(0, 0, 0, 0);
                    if (rr < rows && c < hd_chunks) {
                        const int tok = rr / p.group, g = rr - tok * p.group;
                        const char *src = p.q + (int64_t)(q0 + tok0 + t * tt + tok) * p.q_token +
                                          (int64_t)(kvh * p.group + g) * p.q_head + c * 16;
                        if (p.q_vec) {
                            v[u] = __ldg(reinterpret_cast<const uint4 *>(src));
                        } else {
                            const uint16_t *e = reinterpret_cast<const uint16_t *>(src);
                            v[u] = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16,
                                              e[4] | (uint32_t)e[5] << 16, e[6] | (uint32_t)e[7] << 16);
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int i = i0 + u * 128, rr = i / kChunks, c = i % kChunks;
                    if (rr < S::kQRows)
                        sts128(smem + t * S::kQBytes + (c >> 3) * (S::kQRows * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4), v[u]);
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_ready);
        }

        const int rows = min(max(toks - t * tt, 0), tt) * p.group;
        if ((warp & 3) * 32 < rows) {  // the warp has rows
            const bool live = r < rows;
            const int tok = tok0 + t * tt + r / p.group, g = r % p.group;
            // keys this row sees, counted from the split's first; a row past the
            // end masks nothing (its result goes nowhere)
            const int64_t seen = p.causal ? max((int64_t)0, min((int64_t)kv, (int64_t)kv - nq + tok + 1)) : kv;
            const int vis = live ? (int)(min(seen, (int64_t)kend) - kbeg) : 0x7fffffff;
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t ts = tmem + lanes + t * kKeyTile, to = tmem + lanes + S::kO + t * DP;
            const float c = p.c;
            float m = -INFINITY;
            float2 l2 = make_float2(0.f, 0.f);
            using PR = Pair<true>;
            bool ok = true;
            for (int j = 0; j < ntiles; ++j) {
                if (!(ok = warp_wait(s_ready + t, (uint32_t)(j & 1)))) break;
                tc_after_sync();
                uint32_t s[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, s[q]);
                tmem_wait_ld();
                const int n = vis - j * kKeyTile;  // keys of this tile the row sees
                if (__any_sync(0xffffffffu, n < kKeyTile)) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (32 * q + i >= n) s[q][i] = 0xff800000u;  // -infinity
                }
                float mx[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const uint32_t *v = &s[q >> 1][16 * (q & 1)];
                    mx[q] = fmaxf(__uint_as_float(v[0]), __uint_as_float(v[1]));
#pragma unroll
                    for (int i = 2; i < 16; i += 2)
                        mx[q] = max3(mx[q], __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                }
                const float mt = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
                const bool grown = mt > m && (m == -INFINITY || (mt - m) * c > kRescale);
                if (__any_sync(0xffffffffu, grown)) {
                    const float mn = grown ? mt : m;
                    const float f = m == -INFINITY ? 0.f : exp2_approx((m - mn) * c);
                    if (j > 0) {
                        // the previous product is in o before it is rescaled
                        if (!(ok = warp_wait(o_done + t, (uint32_t)((j - 1) & 1)))) break;
                        tc_after_sync();
                        const float2 f2 = make_float2(f, f);
#pragma unroll
                        for (int d = 0; d < DP; d += 16) {
                            uint32_t o[16];
                            tmem_ld16(to + d, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                const float2 v = PR::mul(make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), f2);
                                o[i] = __float_as_uint(v.x);
                                o[i + 1] = __float_as_uint(v.y);
                            }
                            tmem_st16(to + d, o);
                        }
                    }
                    l2 = PR::mul(l2, make_float2(f, f));
                    m = mn;
                }
                const float mc = m == -INFINITY ? 0.f : -m * c;
                const float2 c2 = make_float2(c, c), m2 = make_float2(mc, mc);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 x = PR::fma(make_float2(__uint_as_float(s[q][2 * i]), __uint_as_float(s[q][2 * i + 1])), c2, m2);
                        x = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                        w[i] = pack_pair<T>(x);
                        s[q][2 * i] = __float_as_uint(x.x);
                        s[q][2 * i + 1] = __float_as_uint(x.y);
                    }
                    tmem_st16(ts + 16 * q, w);
                    if (q & 1) {
                        // half of p is there: its product can start
                        tmem_wait_st();
                        tc_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive((q == 1 ? p_half : p_ready) + t);
                    }
                }
                // the sum, off the path that the products wait for
                float2 a2[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    a2[q] = make_float2(__uint_as_float(s[q][0]), __uint_as_float(s[q][1]));
#pragma unroll
                    for (int i = 2; i < 32; i += 2)
                        a2[q] = PR::add(a2[q], make_float2(__uint_as_float(s[q][i]), __uint_as_float(s[q][i + 1])));
                }
                l2 = PR::add(l2, PR::add(PR::add(a2[0], a2[1]), PR::add(a2[2], a2[3])));
            }
            // ------------------------------------------------------ results
            if (ok && ntiles > 0) {
                ok = warp_wait(o_done + t, (uint32_t)((ntiles - 1) & 1));
                tc_after_sync();
            }
            if (ok) {
                const float l = l2.x + l2.y;
                const bool none = m == -INFINITY && !(l != l);  // no key seen
                const float inv = none ? 0.f : 1.f / l;
                const float lse2 = none ? -INFINITY : m * c + log2f(l);
                const int64_t token = q0 + tok;
                const int head = kvh * p.group + g;
                const int64_t orow = token * p.heads + head;
                if (live && p.splits > 1) p.part_lse[(int64_t)split * p.tokens * p.heads + orow] = lse2;
                if (live && p.splits == 1 && p.lse) p.lse[orow] = lse2 * 0.693147180559945309f;
                float *po = p.splits > 1 ? p.part_o + ((int64_t)split * p.tokens * p.heads + orow) * p.head_dim : nullptr;
                char *out = p.out + token * p.out_token + (int64_t)head * p.out_head;
#pragma unroll
                for (int d = 0; d < DP; d += 32) {
                    if (d >= p.head_dim) break;
                    uint32_t o[32];
                    if (ntiles > 0) {
                        __syncwarp();
                        tmem_ld32(to + d, o);
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = none ? 0u : __float_as_uint(__uint_as_float(o[i]) * inv);
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        if (!live || d + i >= p.head_dim) continue;
                        if (p.splits > 1) {
                            reinterpret_cast<uint4 *>(po + d + i)[0] = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                            reinterpret_cast<uint4 *>(po + d + i)[1] = make_uint4(o[i + 4], o[i + 5], o[i + 6], o[i + 7]);
                            continue;
                        }
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = pack_pair<T>(make_float2(__uint_as_float(o[i + 2 * k]), __uint_as_float(o[i + 2 * k + 1])));
                        char *dst = out + (d + i) * 2;
                        if (p.out_vec) {
                            *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
                        } else {
                            uint16_t *d16 = reinterpret_cast<uint16_t *>(dst);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                d16[2 * k] = (uint16_t)w[k];
                                d16[2 * k + 1] = (uint16_t)(w[k] >> 16);
                            }
                        }
                    }
                }
            }
        }
    }
    __syncwarp();
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    if (warp == kIssuer) {
        __syncwarp();
        tmem_dealloc(tmem, S::kCols);
    }
}

// The splits of a row joined: o = sum_s 2^(lse_s - M) o_s / sum_s 2^(lse_s - M),
// in the splits' order. One warp a row; 8 values a lane and step.
template <typename T>
__global__ void __launch_bounds__(128) paged_attn_join(const __grid_constant__ AttnParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    // unit = (sequence, its token up to max_q, head)
    const int64_t per_seq = (int64_t)p.max_q * p.heads;
    if (unit >= per_seq * p.batch) return;
    const int b = (int)(unit / per_seq);
    const int64_t rest = unit - b * per_seq;
    const int tok = (int)(rest / p.heads), head = (int)(rest - (int64_t)tok * p.heads);
    const int T_ = (int)p.tokens;
    const int q0 = min(max(__ldg(p.cu_q + b), 0), T_);
    const int nq = min(max(__ldg(p.cu_q + b + 1), q0), T_) - q0;
    if (tok >= nq) return;
    const int kv = max(0, min(min(__ldg(p.kv_lens + b), p.max_kv), (int)min((int64_t)p.width * p.page_size, (int64_t)0x7fffffff)));
    const int64_t seen = p.causal ? max((int64_t)0, min((int64_t)kv, (int64_t)kv - nq + tok + 1)) : kv;
    const int n = (int)((seen + p.chunk - 1) / p.chunk);  // splits that hold keys of this row
    const int64_t token = q0 + tok, orow = token * p.heads + head, plane = p.tokens * p.heads;
    float top = -INFINITY;
    bool bad = false;
    for (int s = lane; s < n; s += 32) {
        const float v = p.part_lse[s * plane + orow];
        bad |= v != v;
        top = fmaxf(top, v);
    }
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (__any_sync(0xffffffffu, bad)) top = NAN;
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    const int e = lane * 4;  // values e .. e + 4 of the row
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < n; ++s) {
        const float w = exp2_approx(p.part_lse[s * plane + orow] - ref);
        sum += w;
        if (e < p.head_dim) {
            const float4 v = *reinterpret_cast<const float4 *>(p.part_o + (s * plane + orow) * p.head_dim + e);
            a[0] = __fmaf_rn(w, v.x, a[0]);
            a[1] = __fmaf_rn(w, v.y, a[1]);
            a[2] = __fmaf_rn(w, v.z, a[2]);
            a[3] = __fmaf_rn(w, v.w, a[3]);
        }
    }
    const bool none = top == -INFINITY;
    const float inv = none ? 0.f : 1.f / sum;
    if (lane == 0 && p.lse) p.lse[orow] = none ? -INFINITY : (top + log2f(sum)) * 0.693147180559945309f;
    if (e < p.head_dim) {
        char *dst = p.out + token * p.out_token + (int64_t)head * p.out_head + e * 2;
        const uint32_t w0 = pack_pair<T>(make_float2(a[0] * inv, a[1] * inv)), w1 = pack_pair<T>(make_float2(a[2] * inv, a[3] * inv));
        if (p.out_vec) {
            *reinterpret_cast<uint2 *>(dst) = make_uint2(w0, w1);
        } else {
            uint16_t *d16 = reinterpret_cast<uint16_t *>(dst);
            d16[0] = (uint16_t)w0;
            d16[1] = (uint16_t)(w0 >> 16);
            d16[2] = (uint16_t)w1;
            d16[3] = (uint16_t)(w1 >> 16);
        }
    }
}

// ------------------------------------------------------------------ host --

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once (the library does not
// link the driver).
static EncodeTiled encoder() {
    static std::mutex mu;
    static EncodeTiled fn = nullptr;
    std::lock_guard<std::mutex> lk(mu);
    if (!fn) {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) == cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiled>(f);
    }
    return fn;
}

static int gcd_of(int a, int b) { return b == 0 ? a : gcd_of(b, a % b); }

struct Three {
    int64_t v[3];
};

// A 4-D array (head_dim and three more dimensions, strides in elements of 2
// bytes) copied in boxes of 64 values by `box1` by 1 by `box3`, swizzled by
// 128 bytes. The cache: (head_dim, place in the page, head, page); q:
// (head_dim, head in the group, key head, token).
static bool tile_map(CUtensorMap *map, int dtype, const void *base, int d, Three n, Three stride, int box1, int box3) {
    EncodeTiled enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)n.v[0], (cuuint64_t)n.v[1], (cuuint64_t)n.v[2]};
    cuuint64_t strides[3];
    // a dimension of one entry has no stride: any legal value serves
    for (int i = 0; i < 3; ++i) strides[i] = (cuuint64_t)(n.v[i] > 1 ? stride.v[i] : d) * 2;
    const cuuint32_t box[4] = {64, (cuuint32_t)box1, 1, (cuuint32_t)box3}, ones[4] = {1, 1, 1, 1};
    return enc(map, dtype == RMSNORM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
               const_cast<void *>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Strides (in elements of 2 bytes) and base that a tiled copy takes: 16-byte
// boundaries everywhere.
static bool tile_stride(int64_t s, int64_t n) { return n <= 1 || (s > 0 && s % 8 == 0 && s < (int64_t)1 << 38); }

// How a call is cut: the geometry, the row tiles and the splits over keys.
struct AttnCut {
    int nq, tile_toks, q_tiles, splits, chunk;
    size_t workspace;
};

static AttnCut attn_cut(const paged_attn_call_t &c, int sms) {
    AttnCut k;
    const int64_t group = c.q_heads / c.cache.heads;
    const int64_t rows = (int64_t)c.max_q * group;
    // few rows: the cache's bytes bound the call, and 64 rows a CTA let two
    // CTAs share an SM
    k.nq = rows <= 64 ? 1 : 2;
    // a row tile takes whole tokens: the tiled copy of q then is one box
    k.tile_toks = (int)((k.nq == 1 ? 64 : 128) / group);
    const int64_t per = (int64_t)k.nq * k.tile_toks;
    k.q_tiles = (int)(((int64_t)c.max_q + per - 1) / per);
    const int64_t ctas = (int64_t)c.batch * c.cache.heads * k.q_tiles;
    const int64_t slots = (int64_t)sms * (k.nq == 1 ? 2 : 1);
    const int64_t tiles = ((int64_t)c.max_kv + kKeyTile - 1) / kKeyTile;
    k.splits = 1;
    k.chunk = 0;
    if (ctas < slots && tiles > 1) {
        int64_t want = slots / ctas;
        const int64_t least = 2;  // key tiles a split is worth
        if (want > tiles / least) want = tiles / least;
        if (want > 1) {
            const int64_t per_split = (tiles + want - 1) / want;
            k.splits = (int)((tiles + per_split - 1) / per_split);
            k.chunk = (int)(per_split * kKeyTile);
        }
    }
    k.workspace = 0;
    if (k.splits > 1) {
        const size_t r = (size_t)c.tokens * c.q_heads * k.splits;
        k.workspace = ((r * c.head_dim * 4 + 255) / 256 + (r * 4 + 255) / 256) * 256;
    }
    return k;
}

// Sizes a call may have (pointers apart).
static rmsnorm_status_t attn_sizes(const paged_attn_call_t &c) {
    if (c.dtype != RMSNORM_BF16 && c.dtype != RMSNORM_F16)
        return c.dtype == RMSNORM_F32 ? RMSNORM_ERR_UNSUPPORTED : RMSNORM_ERR_INVALID_ARG;
    if (c.head_dim < 1 || c.batch < 0 || c.tokens < 0 || c.tokens > 0x7fffffffLL || c.q_heads < 1 ||
        c.cache.heads < 1 || c.q_heads % c.cache.heads != 0 || c.max_q < 0 || c.max_kv < 0 || c.table_width < 0)
        return RMSNORM_ERR_INVALID_ARG;
    if (c.head_dim % 8 != 0 || c.head_dim > 128 || c.q_heads / c.cache.heads > 128) return RMSNORM_ERR_UNSUPPORTED;
    if ((int64_t)c.max_q * (c.q_heads / c.cache.heads) > 0x3fffffffLL) return RMSNORM_ERR_UNSUPPORTED;
    return RMSNORM_SUCCESS;
}

template <typename T, int DP, int NQ>
static int launch_attn(const AttnParams &p, const CUtensorMap (&maps)[3], unsigned grid, cudaStream_t stream) {
    using S = AttnShape<DP, NQ>;
    auto *kernel = paged_attn<T, DP, NQ>;
    const int e = allow_staged_smem(reinterpret_cast<const void *>(kernel));
    if (e != 0) return e;
    LaunchCfg lc(grid, S::kThreads, S::kSmem, stream);
    return (int)cudaLaunchKernelEx(&lc.cfg, kernel, p, maps[0], maps[1], maps[2]);
}

template <typename T>
static int launch_attn_t(int nq, const AttnParams &p, const CUtensorMap (&maps)[3], unsigned grid, cudaStream_t s) {
    if (p.head_dim > 64)
        return nq == 2 ? launch_attn<T, 128, 2>(p, maps, grid, s) : launch_attn<T, 128, 1>(p, maps, grid, s);
    return nq == 2 ? launch_attn<T, 64, 2>(p, maps, grid, s) : launch_attn<T, 64, 1>(p, maps, grid, s);
}

static rmsnorm_status_t attn_impl(const paged_attn_call_t &c, cudaStream_t stream) {
    rmsnorm_status_t st = attn_sizes(c);
    if (st != RMSNORM_SUCCESS) return st;
    if (!std::isfinite(c.scale) || c.scale <= 0.f) return RMSNORM_ERR_INVALID_ARG;
    const paged_cache_t &pc = c.cache;
    if (pc.page_size < 1 || pc.pages < 0 || pc.pages > 0x7ffffffeLL) return RMSNORM_ERR_INVALID_ARG;
    if (pc.page_size % 8 != 0) return RMSNORM_ERR_UNSUPPORTED;
    if (c.workspace && !on(c.workspace, 16)) return RMSNORM_ERR_WORKSPACE;
    if (c.tokens == 0 || c.batch == 0 || c.max_q == 0) return RMSNORM_SUCCESS;
    if (!c.q || !c.out || !on(c.q, 2) || !on(c.out, 2) || !on(c.lse, 4) || !c.kv_lens || !c.cu_q ||
        !on(c.block_table, 4) || !on(c.kv_lens, 4) || !on(c.cu_q, 4))
        return RMSNORM_ERR_INVALID_ARG;
    // without a page every sequence is empty; the kernel then reads no table
    const bool empty = pc.pages == 0 || c.table_width == 0 || c.max_kv == 0;
    if (!empty && (!pc.k || !pc.v || !c.block_table)) return RMSNORM_ERR_INVALID_ARG;

    auto legal = [&](const void *base, int64_t page, int64_t slot, int64_t head) {
        return on(base, 16) && tile_stride(page, pc.pages) && tile_stride(slot, pc.page_size) && tile_stride(head, pc.heads);
    };
    if (!empty && (!legal(pc.k, pc.k_page, pc.k_slot, pc.k_head) || !legal(pc.v, pc.v_page, pc.v_slot, pc.v_head)))
        return RMSNORM_ERR_UNSUPPORTED;

    int sms = 0, *status = nullptr;
    int e = current_device(&sms, &status);
    if (e != 0) return head_cuda_fail(e);
    paged_attn_call_t cc = c;
    if (empty) cc.max_kv = 0;
    const AttnCut cut = attn_cut(cc, sms);

    AttnParams p;
    std::memset(&p, 0, sizeof p);
    CUtensorMap maps[3];  // q, k, v
    std::memset(maps, 0, sizeof maps);
    p.box_rows = gcd_of(pc.page_size, kKeyTile);
    if (!empty) {
        const int b = p.box_rows;
        if (!tile_map(&maps[1], c.dtype, pc.k, c.head_dim, {pc.page_size, pc.heads, pc.pages}, {pc.k_slot, pc.k_head, pc.k_page}, b, 1) ||
            !tile_map(&maps[2], c.dtype, pc.v, c.head_dim, {pc.page_size, pc.heads, pc.pages}, {pc.v_slot, pc.v_head, pc.v_page}, b, 1))
            return RMSNORM_ERR_UNSUPPORTED;
    }

    void *ws = c.workspace;
    bool owned = false;
    if (cut.workspace > 0) {
        if (ws) {
            if (c.workspace_bytes < cut.workspace) return RMSNORM_ERR_WORKSPACE;
        } else {
            const cudaError_t me = cudaMallocAsync(&ws, cut.workspace, stream);
            if (me != cudaSuccess) return head_cuda_fail((int)me);
            owned = true;
        }
        const size_t r = (size_t)c.tokens * c.q_heads * cut.splits;
        p.part_o = static_cast<float *>(ws);
        p.part_lse = reinterpret_cast<float *>(static_cast<char *>(ws) + (r * c.head_dim * 4 + 255) / 256 * 256);
    }
    p.q = static_cast<const char *>(c.q);
    p.out = static_cast<char *>(c.out);
    p.lse = c.lse;
    p.table = c.block_table;
    p.kv_lens = c.kv_lens;
    p.cu_q = c.cu_q;
    p.q_token = stride_of(c.q_token, c.tokens) * 2;
    p.q_head = stride_of(c.q_head, c.q_heads) * 2;
    p.out_token = stride_of(c.out_token, c.tokens) * 2;
    p.out_head = stride_of(c.out_head, c.q_heads) * 2;
    p.table_stride = stride_of(c.table_stride, c.batch);
    p.tokens = c.tokens;
    p.status = status;
    p.c = c.scale * 1.44269504088896340736f;
    p.batch = c.batch;
    p.width = empty ? 0 : c.table_width;
    p.heads = c.q_heads;
    p.kv_heads = pc.heads;
    p.group = c.q_heads / pc.heads;
    p.head_dim = c.head_dim;
    p.pages = (int)pc.pages;
    p.page_size = pc.page_size;
    p.max_q = c.max_q;
    p.max_kv = cc.max_kv;
    p.causal = c.causal != 0;
    p.q_tiles = cut.q_tiles;
    p.splits = cut.splits;
    p.chunk = cut.chunk;
    p.tile_toks = cut.tile_toks;
    // (a group's heads share a box: their stride counts even for one key head)
    if (!empty && on(c.q, 16) && tile_stride(c.q_head, c.q_heads) && tile_stride(c.q_token, c.tokens))
        p.q_tma = tile_map(&maps[0], c.dtype, c.q, c.head_dim, {p.group, pc.heads, c.tokens},
                           {c.q_head, c.q_head * p.group, c.q_token}, p.group, p.tile_toks);
    p.q_vec = on(c.q, 16) && p.q_token % 16 == 0 && p.q_head % 16 == 0;
    p.out_vec = on(c.out, 16) && p.out_token % 16 == 0 && p.out_head % 16 == 0;

    const int64_t grid = (int64_t)c.batch * pc.heads * cut.q_tiles * cut.splits;
    const int64_t join = ((int64_t)c.batch * c.max_q * c.q_heads + 3) / 4;
    int le = 0;
    if (grid > 0x7fffffffLL || join > 0x7fffffffLL) {
        st = RMSNORM_ERR_UNSUPPORTED;
    } else {
        le = c.dtype == RMSNORM_BF16 ? launch_attn_t<__nv_bfloat16>(cut.nq, p, maps, (unsigned)grid, stream)
                                     : launch_attn_t<__half>(cut.nq, p, maps, (unsigned)grid, stream);
        if (le == 0 && cut.splits > 1) {
            LaunchCfg lc((unsigned)join, 128, 0, stream);
            le = c.dtype == RMSNORM_BF16 ? (int)cudaLaunchKernelEx(&lc.cfg, paged_attn_join<__nv_bfloat16>, p)
                                         : (int)cudaLaunchKernelEx(&lc.cfg, paged_attn_join<__half>, p);
        }
    }
    if (owned) {
        const cudaError_t fe = cudaFreeAsync(ws, stream);
        if (le == 0 && fe != cudaSuccess) le = (int)fe;
    }
    if (le != 0) return head_cuda_fail(le);
    return st;
}

}  // namespace rmsn

using namespace rmsn;

extern "C" rmsnorm_status_t paged_attn_fwd(const paged_attn_call_t *call, rmsnorm_stream_t stream) {
    if (!call) return RMSNORM_ERR_INVALID_ARG;
    return attn_impl(*call, (cudaStream_t)stream);
}

extern "C" size_t paged_attn_workspace_bytes(const paged_attn_call_t *call) {
    if (!call || attn_sizes(*call) != RMSNORM_SUCCESS) return 0;
    if (call->tokens == 0 || call->batch == 0 || call->max_q == 0) return 0;
    int sms = 0;
    if (current_device(&sms, nullptr) != 0) return 0;
    return attn_cut(*call, sms).workspace;
}
