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
// Geometries (NQ row tiles a CTA):
//  NQ = 2, prompts and chunks: two tiles of 128 rows, one CTA an SM. While the
//    softmax of one tile runs, the other tile's two products do. Bound by the
//    matrix instructions and, over seconds, the power limit: 4864 tokens of 32
//    heads over 32768 keys, D 128, run at 1.82 PFLOP/s (a library product of
//    8192^3: 1.89 in a burst, 1.72 sustained), prompts of 2 x 8192 at 1.54 to
//    1.69. A key tile's shared-memory traffic (q and k read by the first
//    product, v by the second, k and v written) fills the same time.
//  NQ = 1, at most 64 rows (decoding): two CTAs an SM, which cover each other's
//    latencies. Bound by the cache's bytes: 64 sequences of 964 to 8192 keys
//    at 6.2 TB/s, of 8192 each at 7.0.
//
// Few items leave SMs idle, so the keys of a row are split: over the CTAs of a
// cluster that joins them in shared memory (NQ = 1, up to 16), or over items
// whose partial results a second kernel joins. One sequence of 4095 keys, 8 key
// heads: 54 us unsplit, 15.4 with the join's kernel, 11.7 as clusters. What
// remains of a small call is latency: the lengths, the table, the first tile,
// two dependent products and the launch, about 10 us together.
//
// Roles: four warps a tile for the softmax (a thread owns a row: no shuffles),
// one to three warps copying K and V tiles (one box a page, or part of a page),
// one warp issuing matrix instructions. s and p share tensor memory (p, as the
// 16-bit A operand of the second product, overwrites s); o accumulates in
// tensor memory.
//
// Rounding: the matrix instruction takes two operands of one 16-bit type, so p
// is rounded to v's (half a step a weight, of either sign); l sums the unrounded
// p in fp32. Against 64 bits the results are then off by 0.0023 (rms, of the
// result, bf16; fp16 0.00026), where rounding the result alone gives 0.0017
// (0.0002). p in two parts would be half as many products again.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "head_rows.h"
#include "tcgen05.cuh"

namespace rmsn {

constexpr int kKeyTile = 128;
constexpr uint32_t kAttnWait = 1u << 22;  // polls of one barrier before a kernel gives up: 6 s (a failed one takes 1.4 us)
constexpr int kClusterMost = 16;           // CTAs of a cluster (over 8: by opt-in)
constexpr int kJoinTiles = 4;              // key tiles that the join's kernel takes as long as
constexpr int kDecodeChunk = 16;           // key tiles of a decoding item, where there are several a CTA
constexpr int kDecodeItems = 32;           // and at most that many items a CTA
constexpr int kAskAhead = 2;              // key tiles before an item's end to ask for the next one at
constexpr float kRescale = 8.f;           // log2 of how far a row's reference maximum may lag

// Division by a number that the host knows, for 0 <= n < 2^31: with l = ceil
// log2 d and m = floor(2^(31 + l) / d) + 1, n m / 2^(31 + l) is off by less
// than 1 / d. (The instruction sequence for a division by a variable is a
// dependent chain of some 150 cycles, and a small call had ten of them on its
// way to the first copy.)
struct Divisor {
    int d;
    uint32_t mul;
    int shift;
    static Divisor of(int d) {
        Divisor r{d, 0, 0};
        int l = 0;
        while (((int64_t)1 << l) < d) ++l;
        if (d > 1) {
            r.mul = (uint32_t)(((uint64_t)1 << (31 + l)) / (uint64_t)d + 1);
            r.shift = l - 1;
        }
        return r;
    }
    __device__ __forceinline__ int quotient(int n) const {
        return d == 1 ? n : (int)(__umulhi((uint32_t)n, mul) >> shift);
    }
    // the remainder; n becomes the quotient
    __device__ __forceinline__ int split(int &n) const {
        const int q = quotient(n), r = n - q * d;
        n = q;
        return r;
    }
};

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
    int batch, width, heads, group, head_dim, pages, page_size, box_rows;
    int max_q, max_kv, causal, q_tiles, splits, chunk;  // chunk: keys a split takes
    int tile_toks;                                      // tokens a row tile takes
    int nq;                                             // row tiles a CTA takes
    int copiers;                                        // warps that copy K and V: 1 or 3
    int by_seq;                                         // items in the order of the sequences' lengths
    int q_tma, q_vec, out_vec;
    int box_log2;  // box_rows = 2^box_log2
    Divisor by_heads, by_batch, by_splits, by_page, by_group;
};

template <int DP, int NQ>
struct AttnShape {
    static constexpr int kHalves = DP / 64;
    static constexpr int kQRows = NQ == 2 ? 128 : 64;  // rows held of a tile
    static constexpr int kQBytes = kQRows * DP * 2;
    static constexpr int kStage = kKeyTile * DP * 2;
    static constexpr int kStages = NQ == 2 ? (DP == 128 ? 5 : 8) : (DP == 128 ? 3 : 6);
    static constexpr int kBars = NQ * kQBytes + kStages * kStage;
    static constexpr int kSmem = kBars + 512;  // barriers, the work items
    // A fourth warpgroup's worth of warps copies (three) and issues matrix
    // instructions (one). NQ == 2 moves registers from it to the softmax warps:
    // 168 a thread at launch, then 2 x 128 x 208 + 128 x 88 = 384 x 168.
    static constexpr int kThreads = NQ * 128 + 128;
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

// A CTA's waits: bounded, and given up by all roles once one of them
// did. Kept short, since there are two dozen of them and the code's way into
// the instruction cache is what a small call spends its time on.
__device__ __forceinline__ bool wait_on(uint64_t *bar, uint32_t parity, volatile int *gave_up, int *status) {
#pragma unroll 1
    for (uint32_t i = 0; !mbar_try_wait_cta(bar, parity);) {
        if ((++i & 15u) == 0 && (i >= kAttnWait || *gave_up)) {
            *gave_up = 1;
            *status = 1;
            return false;
        }
    }
    return true;
}

// A place in the ring of K and V tiles (K_0, V_0, K_1, ... over all items) and
// the parity of its turn.
template <int NST> struct Ring {
    int st = 0;
    uint32_t turn = 0;
    __device__ __forceinline__ Ring next() const {
        Ring r;
        r.st = st + 1 == NST ? 0 : st + 1;
        r.turn = st + 1 == NST ? turn ^ 1u : turn;
        return r;
    }
};

// One piece of work: a row tile pair (or tile) of a sequence and key head, and
// its keys. Made by the copying warp, read by the others from shared memory.
struct Item {
    int q0, nq, kv;      // the sequence: first row, new tokens, cached tokens
    int tok0, toks;      // its tokens taken here
    int kbeg, kend;      // keys taken here
    int kvh, split, b;
    int parts;           // the rows' keys are split: partial results
    int ntiles;          // key tiles; -1: no more work
    int fix;             // the last tile's values past the sequence's end to become zeros
};

__device__ __forceinline__ int kv_length(const AttnParams &p, int len) {
    return max(0, min(min(len, p.max_kv), (int)min((int64_t)p.width * p.page_size, (int64_t)0x7fffffff)));
}

// Keys that the last row of a row tile sees: tokens up to `end` of the nq new
// ones of a sequence of kv.
__device__ __forceinline__ int keys_seen(const AttnParams &p, int kv, int nq, int end) {
    return p.causal ? (int)min((int64_t)kv, max((int64_t)0, (int64_t)kv - nq + end)) : kv;
}

// Work item `id`, for a whole warp; false: it has nothing to do. The long ones
// come first, since the last to start decide when the call ends: (sequence,
// key head) fastest, then the split, then the row tile from the last rows
// (most keys) on; or, where the keys before the new tokens are most of them,
// by_seq (at most 32 sequences): the sequences from the longest on, in each
// the row tiles, splits and key heads.
template <bool CL>
__device__ __forceinline__ bool decode_item(const AttnParams &p, int id, int per, Item &w) {
    const int lane = threadIdx.x & 31;
    const int T_ = (int)p.tokens;
    int rank = 0;
    if (CL) {  // (the split fastest: a cluster's CTAs)
        rank = p.by_splits.split(id);
    }
    w.kvh = p.by_heads.split(id);
    int b, qt;
    if (CL) {
        b = id;
        qt = 0;
        w.split = rank;
    } else if (p.by_seq) {
        int n = 0, parts = 1, kv = -1;
        if (lane < p.batch) {
            const int c0 = min(max(p.cu_q[lane], 0), T_), c1 = min(max(p.cu_q[lane + 1], c0), T_);
            kv = kv_length(p, p.kv_lens[lane]);
            n = (min(c1 - c0, p.max_q) + per - 1) / per;
            if (p.splits > 1) parts = max((kv + p.chunk - 1) / p.chunk, 1);
        }
        int before = 0;
        for (int o = 0; o < p.batch; ++o) {
            const int k = __shfl_sync(0xffffffffu, kv, o), m = __shfl_sync(0xffffffffu, n * parts, o);
            if (k > kv || (k == kv && o < lane)) before += m;
        }
        const uint32_t mine = __ballot_sync(0xffffffffu, id >= before && id < before + n * parts);
        if (mine == 0) return false;
        b = __ffs((int)mine) - 1;
        id -= __shfl_sync(0xffffffffu, before, b);
        parts = __shfl_sync(0xffffffffu, parts, b);
        qt = __shfl_sync(0xffffffffu, n, b) - 1 - id / parts;
        w.split = id % parts;
    } else {
        b = p.by_batch.split(id);
        w.split = p.by_splits.split(id);
        qt = p.q_tiles - 1 - id;
    }
    w.b = b;
    const int c0 = p.cu_q[b], c1 = p.cu_q[b + 1];
    w.kv = kv_length(p, p.kv_lens[b]);
    w.q0 = min(max(c0, 0), T_);
    w.nq = min(max(c1, w.q0), T_) - w.q0;
    w.tok0 = qt * per;
    w.toks = min(min(w.nq, p.max_q) - w.tok0, per);
    w.parts = 0;
    w.ntiles = 0;
    w.fix = 0;
    if (w.toks <= 0) return CL;
    const int lim = keys_seen(p, w.kv, w.nq, w.tok0 + w.toks);
    w.kbeg = 0;
    w.kend = lim;
    if (p.splits > 1) {
        const int64_t kbeg = (int64_t)w.split * p.chunk;
        if (kbeg >= lim) return CL;  // (rows without keys are the join's)
        w.kbeg = (int)kbeg;
        w.kend = (int)min((int64_t)lim, kbeg + p.chunk);
        w.parts = lim > p.chunk;
    }
    w.ntiles = (w.kend - w.kbeg + kKeyTile - 1) / kKeyTile;
    const int last_valid = w.kv - (w.kbeg + (w.ntiles - 1) * kKeyTile);
    w.fix = w.ntiles > 0 && last_valid < kKeyTile && (last_valid & (p.box_rows - 1)) != 0;
    return true;
}

// A 4 by 4 transposition within groups of four lanes: lane i's c[k] becomes
// lane k's c[i].
__device__ __forceinline__ void swap_lanes(uint32_t &a, uint32_t &b, bool upper, int o) {
    const uint32_t give = upper ? a : b;
    const uint32_t got = __shfl_xor_sync(0xffffffffu, give, o);
    a = upper ? got : a;
    b = upper ? b : got;
}
__device__ __forceinline__ void transpose4(uint4 (&c)[4], int lane) {
    const bool u1 = lane & 1, u2 = lane & 2;
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
        swap_lanes(c[k].x, c[k + 1].x, u1, 1);
        swap_lanes(c[k].y, c[k + 1].y, u1, 1);
        swap_lanes(c[k].z, c[k + 1].z, u1, 1);
        swap_lanes(c[k].w, c[k + 1].w, u1, 1);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        swap_lanes(c[k].x, c[k + 2].x, u2, 2);
        swap_lanes(c[k].y, c[k + 2].y, u2, 2);
        swap_lanes(c[k].z, c[k + 2].z, u2, 2);
        swap_lanes(c[k].w, c[k + 2].w, u2, 2);
    }
}

__device__ __forceinline__ void prefetch_l1(const void *p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

// 32 columns of a tile's scores; columns from n on are masked.
__device__ __forceinline__ void load_scores(uint32_t from, int n, bool masks, uint32_t (&s)[32]) {
    __syncwarp();
    tmem_ld32(from, s);
    tmem_wait_ld();
    if (masks) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i >= n) s[i] = 0xff800000u;  // -infinity
    }
}

// 16 bytes to rows off 16-byte boundaries (out of line: rarely taken).
__device__ __noinline__ void store_halves(uint16_t *to, uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        to[2 * i] = (uint16_t)w[i];
        to[2 * i + 1] = (uint16_t)(w[i] >> 16);
    }
}

// 4 and 16 bytes of another CTA of the cluster, at the address of a variable
// of this one.
__device__ __forceinline__ float ld_cluster(const float *local, uint32_t cta) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(cta));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster4(const void *local, uint32_t cta) {
    uint32_t a;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(cta));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

// o = sum_s 2^(lse_s - M) o_s / sum_s 2^(lse_s - M) over the cluster's CTAs, in
// their order; four values a thread, the rows' chunks dealt to the CTAs.
template <typename T, int DP>
__device__ __forceinline__ void join_cluster(const AttnParams &p, const Item &w, const uint8_t *rows, const float *lse) {
    const int chunks = p.head_dim / 4, total = w.toks * p.group * chunks;
    const int rank = (int)cluster_ctarank(), splits = p.splits;
    for (int i = rank * (int)blockDim.x + (int)threadIdx.x; i < total; i += splits * (int)blockDim.x) {
        const int r = i / chunks, c = i - r * chunks;
        float l[kClusterMost], top = -INFINITY, sum = 0.f;
        float4 v[kClusterMost];
#pragma unroll
        for (int s = 0; s < kClusterMost; ++s) {
            if (s >= splits) break;
            l[s] = ld_cluster(lse + r, (uint32_t)s);
            v[s] = ld_cluster4(rows + r * (DP * 4) + ((c + r) % (DP / 4)) * 16, (uint32_t)s);
        }
#pragma unroll
        for (int s = 0; s < kClusterMost; ++s) {
            if (s >= splits) break;
            top = l[s] != l[s] || top != top ? NAN : fmaxf(top, l[s]);
        }
        const bool none = top == -INFINITY;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int s = 0; s < kClusterMost; ++s) {
            if (s >= splits) break;
            const float e = exp2_approx(l[s] - (none ? 0.f : top));
            sum += e;
            a.x = __fmaf_rn(e, v[s].x, a.x);
            a.y = __fmaf_rn(e, v[s].y, a.y);
            a.z = __fmaf_rn(e, v[s].z, a.z);
            a.w = __fmaf_rn(e, v[s].w, a.w);
        }
        const float inv = none ? 0.f : __fdividef(1.f, sum);
        const int tok = p.by_group.quotient(r);
        const int64_t token = w.q0 + w.tok0 + tok;
        const int head = w.kvh * p.group + r - tok * p.group;
        if (c == 0 && p.lse)
            p.lse[token * p.heads + head] = none ? -INFINITY : (top + __log2f(sum)) * 0.693147180559945309f;
        char *dst = p.out + token * p.out_token + (int64_t)head * p.out_head + c * 8;
        const uint32_t w0 = pack_pair<T>(make_float2(a.x * inv, a.y * inv)), w1 = pack_pair<T>(make_float2(a.z * inv, a.w * inv));
        if (p.out_vec) {
            *reinterpret_cast<uint2 *>(dst) = make_uint2(w0, w1);
        } else {
            uint16_t *e = reinterpret_cast<uint16_t *>(dst);
            e[0] = (uint16_t)w0;
            e[1] = (uint16_t)(w0 >> 16);
            e[2] = (uint16_t)w1;
            e[3] = (uint16_t)(w1 >> 16);
        }
    }
}

// Persistent: a CTA takes its own block's item, then those of blocks that have
// not started (the hardware's order, so the load balances itself), and the
// roles run from one item into the next: while the softmax warps write an
// item's rows, the next one's keys arrive and its first product is done.
// CL (NQ == 1): the splits of a sequence and key head are a cluster. Each CTA
// leaves its rows in its shared memory, and the cluster joins them there: no
// workspace and no second kernel. No CTA takes a second item.
template <typename T, int DP, int NQ, bool CL>
__global__ void __launch_bounds__(NQ * 128 + 128, NQ == 2 ? 1 : 2)
    paged_attn(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap qmap,
               const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using S = AttnShape<DP, NQ>;
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int NST = S::kStages;
    constexpr int kProducer = NQ * 4, kIssuer = NQ * 4 + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::kBars);
    uint64_t *full = bars, *empty = bars + NST;
    uint64_t *s_ready = empty + NST, *p_half = s_ready + NQ, *p_ready = p_half + NQ, *o_done = p_ready + NQ;
    uint64_t *q_ready = o_done + NQ, *q_free = q_ready + 1, *v_fixed = q_free + 1, *drained = v_fixed + 2;
    uint64_t *item_full = drained + 1, *item_empty = item_full + 2, *answered = item_empty + 2;
    static_assert(2 * S::kStages + 4 * NQ + 10 <= 36, "barriers");
    uint8_t *after = smem + S::kBars + 36 * 8;
    void *answer = after;  // 16 bytes, 16-byte aligned
    Item *items = reinterpret_cast<Item *>(after + 16);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(items + 2);
    volatile int *gave_up = reinterpret_cast<volatile int *>(tmem_slot + 1);
    static_assert(36 * 8 + 16 + 2 * sizeof(Item) + 8 <= S::kSmem - S::kBars, "shared memory");

    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int t = 0; t < NQ; ++t) {
            mbar_init(s_ready + t, 1);
            mbar_init(p_half + t, 4);  // the tile's warps
            mbar_init(p_ready + t, 4);
            mbar_init(o_done + t, 1);
        }
        mbar_init(q_ready, p.q_tma ? 1 : NQ * 4);
        mbar_init(q_free, 1);
        mbar_init(drained, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(v_fixed + i, 1);
            mbar_init(item_full + i, 1);
            mbar_init(item_empty + i, NQ * 4 + p.copiers);  // all warps but the one that makes the items
        }
        mbar_init(answered, 1);
        *gave_up = 0;
        mbar_init_fence();
    }
    if (warp == kProducer && lane == 0) {
        prefetch_map(&qmap);
        prefetch_map(&kmap);
        prefetch_map(&vmap);
    }
    // (What the kernel before wrote is read with plain loads and copies only: the
    // non-coherent path wants data that nothing writes while the kernel runs.)
    pdl_wait();
    pdl_trigger();
    if ((smem_u32(smem) & 1023u) != 0) {  // the swizzle goes by the address
        if (threadIdx.x == 0) *p.status = 1;
        return;
    }
    if (warp == kIssuer) tmem_alloc(tmem_slot, S::kCols);
    if (warp == kProducer) {  // the first item's lengths, on their way while the CTA meets
        int b = blockIdx.x;
        if (CL) b = p.by_splits.quotient(b);
        b = p.by_heads.quotient(b);
        b = p.by_seq ? min(lane, p.batch - 1) : p.by_batch.split(b);
        prefetch_l1(p.cu_q + b);
        prefetch_l1(p.cu_q + b + 1);
        prefetch_l1(p.kv_lens + b);
    }
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = *tmem_slot;
    // By a whole warp: all of it goes on or none. The first poll is apart and its
    // branch uniform: as part of the loop, whose lanes may leave one by one, a
    // wait for what is already there cost the inner loop 20% (prompt of 4864
    // tokens over 32768: 1631 -> 1331 us). Every lane polls, and so acquires.
    auto warp_wait = [&](uint64_t *bar, uint32_t parity) {
        if (__all_sync(0xffffffffu, mbar_try_wait_cta(bar, parity))) return true;
        return __all_sync(0xffffffffu, wait_on(bar, parity, gave_up, p.status)) != 0;
    };
    volatile int still = 0;  // the last waits, after giving up, have a limit of their own
    const uint32_t sbase = smem_u32(smem);
    const uint32_t stage0 = sbase + NQ * S::kQBytes;
    const int tt = p.tile_toks;
    // CL: the rows' partial results, over the ring's stages
    uint8_t *join_at = smem + NQ * S::kQBytes;
    float *join_lse = reinterpret_cast<float *>(join_at + S::kQRows * DP * 4);
    static_assert(!CL || S::kQRows * (DP * 4 + 4) <= S::kStages * S::kStage, "join");

    // The n-th item of this CTA, as the producer left it; false: given up.
    auto take = [&](int n, Item &w) {
        if (!warp_wait(item_full + (n & 1), (uint32_t)((n >> 1) & 1))) return false;
        w = items[n & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(item_empty + (n & 1));
        return true;
    };

    if (warp >= kProducer) {
    if constexpr (NQ == 2) fewer_registers<88>();
    // Copies of K and V. A tile is 128 / box_rows boxes by 64 columns. Issuing
    // them takes a warp 85 cycles each (the operands of each lane go through
    // uniform registers): with pages of 8, 5400 cycles a K and V tile where the
    // products take 2100. With small boxes three warps share them; with large
    // ones the other two only cost (2 x 8192 tokens, D 128: pages of 8 1178 ->
    // 707 us and of 16 775 -> 674, but of 64 649 -> 677).
    const int copier = warp == kProducer ? 0 : warp - kIssuer;  // 0, 1, 2
    const int boxes_log2 = 7 - p.box_log2;  // of a key tile's 128 rows
    const int item_box = copier + p.copiers * lane;
    const int piece = item_box & ((1 << boxes_log2) - 1), half = item_box >> boxes_log2;
    const bool copies = half < S::kHalves;
    const uint32_t off = (uint32_t)(half * kKeyTile * 128 + (piece << p.box_log2) * 128);
    // (the table's entry is checked where it is used, a tile later: until then
    // its load is under way)
    auto find = [&](const Item &i, int tile, int &pg, int &pl) {
        const int key = i.kbeg + tile * kKeyTile + (piece << p.box_log2);
        pg = -1;
        pl = 0;
        if (copies && tile < i.ntiles && key < i.kv) {
            const int col = p.by_page.quotient(key);
            pg = p.table[i.b * p.table_stride + col];
            pl = key - col * p.page_size;
        }
    };
    Ring<NST> at;  // the next tile's place
    // This warp's boxes of the next tile, once its place is free.
    auto copy_tile = [&](const CUtensorMap *map, int kvh, int pg, int pl) {
        const int st = at.st;
        if (!warp_wait(empty + st, at.turn ^ 1u)) return false;
        if (copier == 0) {  // (boxes counted before this only wait for it)
            if (lane == 0) mbar_arrive_expect_tx(full + st, S::kStage);
            __syncwarp();
        }
        // what is no page lies outside the cache: zeros
        if ((uint32_t)pg >= (uint32_t)p.pages) {
            pg = p.pages;
            pl = 0;
        }
        if (copies) tile_g2s(stage0 + st * S::kStage + off, map, half * 64, pl, kvh, pg, full + st);
        at = at.next();
        return true;
    };
    if (warp == kProducer) {
        // ------------------------------------------ the work, and its copies
        Item w;
        int page, place;
        int asked = 0;
        bool ok = true;
        auto ask = [&]() {
            if (lane == 0) {
                // (the answer before, read by this warp, precedes the next in its place)
                fence_async_smem();
                mbar_arrive_expect_tx(answered, 16);
                next_block_ask(answer, answered);
            }
            __syncwarp();
            ++asked;
        };
        // The next item with work (this block's own, then those asked for), its
        // first tile looked up; ntiles -1: none.
        int n = 0;  // items
        auto find_next = [&](Item &i, int &pg, int &pl) {
#pragma unroll 1
            for (;; ask()) {
                int id = blockIdx.x;
                if (CL && n > 0) id = -1;
                if (asked > 0) {
                    if (!warp_wait(answered, (uint32_t)((asked - 1) & 1))) {
                        ok = false;
                        break;
                    }
                    id = next_block_answer(answer);
                    __syncwarp();
                }
                if (id < 0) break;
                if (decode_item<CL>(p, id, NQ * tt, i)) {
                    find(i, 0, pg, pl);
                    return;
                }
            }
            i.ntiles = -1;
        };
        // Values past the sequence's end in its last page would meet a zero
        // weight, and 0 * NaN is NaN: they become zeros once the tile is there.
        // (Two barriers in turn: with the items' two places this warp may mend the
        // next item's values before the products of this one's, and no further.)
        Ring<NST> fix_at;
        int fix_from = -1, fixes = 0;
        auto fix_values = [&]() {
            const int st = fix_at.st;
            if (!warp_wait(full + st, fix_at.turn)) {
                ok = false;
                return;
            }
            const int end = ((fix_from >> p.box_log2) + 1) << p.box_log2;  // later boxes are zeros
            const int chunks = (end - fix_from) * 8;
#pragma unroll 1
            for (int i = lane; i < chunks * S::kHalves; i += 32) {
                const int h = i / chunks, c = i - h * chunks;
                sts128(smem + NQ * S::kQBytes + st * S::kStage + h * kKeyTile * 128 + fix_from * 128 + c * 16,
                       make_uint4(0, 0, 0, 0));
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(v_fixed + (fixes & 1));
            ++fixes;
            fix_from = -1;
        };

        int q_loads = 0;
#pragma unroll 1
        for (;; ++n) {
            find_next(w, page, place);
            if (!ok) break;
            if (n >= 2 && !warp_wait(item_empty + (n & 1), (uint32_t)(((n >> 1) - 1) & 1))) break;
            // (an item that copies nothing leaves nothing to put the mending off to;
            // behind the wait, which keeps it within the two barriers)
            if (w.ntiles <= 0 && fix_from >= 0) fix_values();
            if (!ok) break;
            if (lane == 0) {
                items[n & 1] = w;
                mbar_arrive(item_full + (n & 1));
            }
            __syncwarp();
            if (w.ntiles < 0) break;
            // The next is asked for when the item's last tiles are being copied:
            // late, so that the blocks left go to whoever is done first, and early
            // enough for the answer (a microsecond) to be there in time.
            const int ask_at = max(2 * (w.ntiles - kAskAhead), 1);
            if (!CL && w.ntiles == 0) ask();
            int next_page, next_place;
            Ring<NST> last_at;
#pragma unroll 1
            for (int i = 0; i < 2 * w.ntiles; ++i) {  // K_0, V_0, K_1, ...
                last_at = at;
                if (!(ok = copy_tile(i & 1 ? &vmap : &kmap, w.kvh, page, place))) break;
                if (i == 0) {
                    // (K_0's place in the ring did not wait for the values mended here)
                    if (fix_from >= 0) fix_values();
                    if (ok && p.q_tma) {
                        // q's rows: tt tokens of `group` heads are one box, row after row
                        if (q_loads > 0 && !warp_wait(q_free, (uint32_t)((q_loads - 1) & 1))) ok = false;
                        if (ok && lane == 0) {
                            const int act = w.toks > tt ? 2 : 1;
                            mbar_arrive_expect_tx(q_ready, (uint32_t)(act * S::kHalves * tt * p.group * 128));
#pragma unroll 1
                            for (int t = 0; t < act; ++t)
#pragma unroll 1
                                for (int h = 0; h < S::kHalves; ++h)
                                    tile_g2s(sbase + t * S::kQBytes + h * (S::kQRows * 128), &qmap, h * 64, 0, w.kvh,
                                             w.q0 + w.tok0 + t * tt, q_ready);
                        }
                        __syncwarp();
                        if (ok) ++q_loads;
                    }
                    if (!ok) break;
                }
                if (i & 1) {
                    page = next_page;
                    place = next_place;
                } else {
                    find(w, (i >> 1) + 1, next_page, next_place);
                }
                if (!CL && i == ask_at) ask();
            }
            if (!ok) break;
            if (w.fix) {
                fix_from = w.kv - (w.kbeg + (w.ntiles - 1) * kKeyTile);
                fix_at = last_at;
            }
        }
        if (*gave_up) {  // no copy may be in flight when the CTA ends
            if (q_loads > 0) wait_on(q_ready, (uint32_t)((q_loads - 1) & 1), &still, p.status);
            // (the last turn of each place: a place not copied to yet has turn 1 behind it)
#pragma unroll 1
            for (int i = 0; i < NST; ++i, at = at.next()) wait_on(full + at.st, at.turn ^ 1u, &still, p.status);
            if (asked > 0) wait_on(answered, (uint32_t)((asked - 1) & 1), &still, p.status);
        }
    } else if (warp != kIssuer) {
        // ---------------------------------------------- the copies' other warps
#pragma unroll 1
        for (int n = 0; copier < p.copiers; ++n) {
            Item w;
            if (!take(n, w) || w.ntiles < 0) break;
            int page, place, next_page, next_place;
            find(w, 0, page, place);
            bool ok = true;
#pragma unroll 1
            for (int i = 0; i < 2 * w.ntiles; ++i) {
                if (!(ok = copy_tile(i & 1 ? &vmap : &kmap, w.kvh, page, place))) break;
                if (i & 1) {
                    page = next_page;
                    place = next_place;
                } else {
                    find(w, (i >> 1) + 1, next_page, next_place);
                }
            }
            if (!ok) break;
        }
        if (copier < p.copiers && *gave_up) {  // the newest place's turn ends when all its copies are there
            Ring<NST> last;
            last.st = at.st == 0 ? NST - 1 : at.st - 1;
            last.turn = at.st == 0 ? at.turn ^ 1u : at.turn;
            wait_on(full + last.st, last.turn, &still, p.status);
        }
    } else {
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
        auto done_with = [&](uint64_t *bar) {
            if (issues) mma_commit(bar);
            __syncwarp();
        };
        auto arrived = [&](const Ring<NST> &r) { return warp_wait(full + r.st, r.turn); };
        Ring<NST> kr;  // the next key tile's place
        uint32_t q_turn = 0, turn[2] = {0, 0};
        int fixes = 0;
        bool ok = true;
#pragma unroll 1
        for (int n = 0; ok; ++n) {
            Item w;
            if (!(ok = take(n, w)) || w.ntiles < 0) break;
            if (w.ntiles == 0) continue;
            const int act = w.toks > tt ? 2 : 1;
            ok = arrived(kr) && warp_wait(q_ready, q_turn);
            if (!ok) break;
            q_turn ^= 1u;
            tc_after_sync();
            // (what the softmax still had to read of s, the products issued before have waited for)
#pragma unroll
            for (int t = 0; t < NQ; ++t)
                if (t < act) qk(t, kr.st);
            done_with(empty + kr.st);
            if (w.ntiles == 1) done_with(q_free);
            Ring<NST> vr = kr.next();
            kr = vr.next();
            ok = arrived(vr);
#pragma unroll 1
            for (int j = 0; j < w.ntiles && ok; ++j) {
                const bool more = j + 1 < w.ntiles;
                if (!more && w.fix) {
                    ok = warp_wait(v_fixed + (fixes & 1), (uint32_t)((fixes >> 1) & 1));
                    ++fixes;
                }
                const Ring<NST> vn = kr.next();  // the next values' place
#pragma unroll
                for (int t = 0; t < NQ; ++t) {
                    if (t >= act || !ok) break;
                    if (!(ok = warp_wait(p_half + t, turn[t]))) break;
                    tc_after_sync();
                    pv(t, vr.st, 0, j > 0);
                    if (!(ok = warp_wait(p_ready + t, turn[t]))) break;
                    turn[t] ^= 1u;
                    tc_after_sync();
                    pv(t, vr.st, 1, true);
                    if (t == act - 1) done_with(empty + vr.st);
                    if (more) {
                        if (t == 0) ok = arrived(kr);
                        if (ok) qk(t, kr.st);
                        // (here, where the products just issued cover the wait)
                        if (ok && t == 0) ok = arrived(vn);
                    }
                }
                if (more && ok) {
                    done_with(empty + kr.st);
                    if (j + 2 == w.ntiles) done_with(q_free);
                    vr = vn;
                    kr = vn.next();
                }
            }
        }
        if (*gave_up) {  // nor may a matrix instruction be
            __syncwarp();
            if (issues) mma_commit(drained);
            wait_on(drained, 0, &still, p.status);
        }
    }
    } else {
        // --------------------------------------------------------- softmax
        if constexpr (NQ == 2) more_registers<208>();
        const int t = warp >> 2, r = threadIdx.x & 127;  // tile, row in it
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + t * kKeyTile, to = tmem + lanes + S::kO + t * DP;
        const int row_tok = p.by_group.quotient(r), row_head = r - row_tok * p.group;
        const float c = p.c;
        using PR = Pair<true>;
        int steps = 0;  // key tiles, over all items
        uint32_t q_turn = 0;
        bool ok = true;
#pragma unroll 1
        for (int n = 0; ok; ++n) {
            Item w;
            if (!(ok = take(n, w)) || w.ntiles < 0) break;
            const int rows = min(max(w.toks - t * tt, 0), tt) * p.group;
            if (w.ntiles > 0 && !p.q_tma) {
                // q that a tiled copy does not take (bases or strides off 16-byte
                // boundaries): eight chunks in flight a thread, to the swizzled rows,
                // zeros past the rows and head_dim. (The item before's last product
                // with q was done before its last softmax.)
                constexpr int kChunks = S::kHalves * 8, kBatch = 8;
                const int hd_chunks = p.head_dim / 8;
#pragma unroll 1
                for (int i0 = r; i0 < S::kQRows * kChunks; i0 += 128 * kBatch) {
                    uint4 v[kBatch];
#pragma unroll
                    for (int u = 0; u < kBatch; ++u) {
                        const int i = i0 + u * 128, rr = i / kChunks, ch = i % kChunks;
                        v[u] = make_uint4(0, 0, 0, 0);
                        if (rr < rows && ch < hd_chunks) {
                            const int tok = p.by_group.quotient(rr), g = rr - tok * p.group;
                            const char *src = p.q + (int64_t)(w.q0 + w.tok0 + t * tt + tok) * p.q_token +
                                              (int64_t)(w.kvh * p.group + g) * p.q_head + ch * 16;
                            if (p.q_vec) {
                                v[u] = *reinterpret_cast<const uint4 *>(src);
                            } else {
                                const uint16_t *e = reinterpret_cast<const uint16_t *>(src);
                                v[u] = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16,
                                                  e[4] | (uint32_t)e[5] << 16, e[6] | (uint32_t)e[7] << 16);
                            }
                        }
                    }
#pragma unroll
                    for (int u = 0; u < kBatch; ++u) {
                        const int i = i0 + u * 128, rr = i / kChunks, ch = i % kChunks;
                        if (rr < S::kQRows)
                            sts128(smem + t * S::kQBytes + (ch >> 3) * (S::kQRows * 128) + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4),
                                   v[u]);
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_ready);
                // all of q is there before any warp goes on: one without rows would
                // arrive for its next item while this one's turn still counts
                if (!(ok = warp_wait(q_ready, q_turn))) break;
                q_turn ^= 1u;
            }
            if (rows == 0) continue;  // (the tile's products are not issued either)
            if ((warp & 3) * 32 >= rows) {
                // a warp without rows only keeps the tile's count of arrivals
#pragma unroll 1
                for (int j = 0; j < w.ntiles; ++j, ++steps) {
                    if (!(ok = warp_wait(s_ready + t, (uint32_t)(steps & 1)))) break;
                    if (lane == 0) {
                        mbar_arrive(p_half + t);
                        mbar_arrive(p_ready + t);
                    }
                }
                continue;
            }
            const bool live = r < rows;
            const int tok = w.tok0 + t * tt + row_tok;
            // keys this row sees, counted from the item's first; a row past the
            // end masks nothing (its result goes nowhere)
            const int64_t seen = p.causal ? max((int64_t)0, min((int64_t)w.kv, (int64_t)w.kv - w.nq + tok + 1)) : w.kv;
            const int vis = live ? (int)(min(seen, (int64_t)w.kend) - w.kbeg) : 0x7fffffff;
            float m = -INFINITY;
            float2 l2 = make_float2(0.f, 0.f);
#pragma unroll 1
            for (int j = 0; j < w.ntiles; ++j, ++steps) {
                if (!(ok = warp_wait(s_ready + t, (uint32_t)(steps & 1)))) break;
                tc_after_sync();
                const int nk = vis - j * kKeyTile;  // keys of this tile the row sees
                const bool masks = __any_sync(0xffffffffu, nk < kKeyTile);
                // NQ == 2 holds the tile's scores in registers; NQ == 1, with fewer
                // of them and time to spare, reads them twice, 32 columns at a time.
                constexpr bool kHold = NQ == 2;
                uint32_t s[kHold ? 4 : 1][32];
                float mt;
                if constexpr (kHold) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, s[q]);
                    tmem_wait_ld();
                    if (masks) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (32 * q + i >= nk) s[q][i] = 0xff800000u;  // -infinity
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
                    mt = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
                } else {
                    mt = -INFINITY;
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        load_scores(ts + 32 * q, nk - 32 * q, masks, s[0]);
                        float mx[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            mx[k] = fmaxf(__uint_as_float(s[0][8 * k]), __uint_as_float(s[0][8 * k + 1]));
#pragma unroll
                            for (int i = 2; i < 8; i += 2)
                                mx[k] = max3(mx[k], __uint_as_float(s[0][8 * k + i]), __uint_as_float(s[0][8 * k + i + 1]));
                        }
                        mt = fmaxf(max3(mt, mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    }
                }
                const bool grown = mt > m && (m == -INFINITY || (mt - m) * c > kRescale);
                if (__any_sync(0xffffffffu, grown)) {
                    const float mn = grown ? mt : m;
                    const float f = m == -INFINITY ? 0.f : exp2_approx((m - mn) * c);
                    if (j > 0) {
                        // the previous product is in o before it is rescaled
                        if (!(ok = warp_wait(o_done + t, (uint32_t)((steps - 1) & 1)))) break;
                        tc_after_sync();
                        const float2 f2 = make_float2(f, f);
#pragma unroll 1
                        for (int d = 0; d < DP; d += 16) {
                            uint32_t o[16];
                            __syncwarp();
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
                if constexpr (kHold) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float2 x = PR::fma(make_float2(__uint_as_float(s[q][2 * i]), __uint_as_float(s[q][2 * i + 1])), c2, m2);
                            x = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                            pk[i] = pack_pair<T>(x);
                            s[q][2 * i] = __float_as_uint(x.x);
                            s[q][2 * i + 1] = __float_as_uint(x.y);
                        }
                        tmem_st16(ts + 16 * q, pk);
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
                } else {
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        load_scores(ts + 32 * q, nk - 32 * q, masks, s[0]);
                        uint32_t pk[16];
                        float2 a2 = make_float2(0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float2 x = PR::fma(make_float2(__uint_as_float(s[0][2 * i]), __uint_as_float(s[0][2 * i + 1])), c2, m2);
                            x = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                            pk[i] = pack_pair<T>(x);
                            a2 = PR::add(a2, x);
                        }
                        l2 = PR::add(l2, a2);
                        // (columns 16 q .. of p lie before the scores still to be read)
                        tmem_st16(ts + 16 * q, pk);
                        if (q & 1) {
                            tmem_wait_st();
                            tc_before_sync();
                            __syncwarp();
                            if (lane == 0) mbar_arrive((q == 1 ? p_half : p_ready) + t);
                        }
                    }
                }
            }
            // ------------------------------------------------------ results
            if (!ok) break;
            auto o_ready = [&]() {
                if (w.ntiles == 0) return true;
                if (!warp_wait(o_done + t, (uint32_t)((steps - 1) & 1))) return false;
                tc_after_sync();
                return true;
            };
            const float l = l2.x + l2.y;
            const bool none = m == -INFINITY && !(l != l);  // no key seen
            const float inv = none ? 0.f : __fdividef(1.f, l);
            const float lse2 = none ? -INFINITY : m * c + __log2f(l);
            if constexpr (CL) {
                // to this CTA's shared memory, whose K and V are done with: a
                // row's 16-byte chunks turned by the row, so that the lanes' stores
                // spread over the banks
                if (!(ok = o_ready())) break;
                if (live) join_lse[r] = lse2;
#pragma unroll 1
                for (int d = 0; d < p.head_dim; d += 32) {
                    uint32_t o[32];
                    if (w.ntiles > 0) {
                        __syncwarp();
                        tmem_ld32(to + d, o);
                        tmem_wait_ld();
                    }
                    if (!live) continue;
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (!none)
                            v = make_uint4(__float_as_uint(__uint_as_float(o[i]) * inv), __float_as_uint(__uint_as_float(o[i + 1]) * inv),
                                           __float_as_uint(__uint_as_float(o[i + 2]) * inv), __float_as_uint(__uint_as_float(o[i + 3]) * inv));
                        sts128(join_at + r * (DP * 4) + (((d + i) / 4 + r) % (DP / 4)) * 16, v);
                    }
                }
                continue;
            }
            const int head = w.kvh * p.group + row_head;
            const int64_t token = w.q0 + tok, orow = token * p.heads + head, plane = p.tokens * p.heads;
            const bool parts = w.parts;
            if (live) {
                if (parts)
                    p.part_lse[(int64_t)w.split * plane + orow] = lse2;
                else if (p.lse)
                    p.lse[orow] = lse2 * 0.693147180559945309f;
            }
            // A row is a lane's, and 16 bytes of each of 32 rows a store would
            // occupy the store path for 32 cycles: four lanes exchange their
            // chunks and write 64 bytes of each of eight rows instead.
            char *dst = parts ? reinterpret_cast<char *>(p.part_o + ((int64_t)w.split * plane + orow) * p.head_dim)
                              : p.out + token * p.out_token + (int64_t)head * p.out_head;
            char *rows4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint64_t a = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(live ? dst : nullptr), (lane & 28) + k);
                rows4[k] = reinterpret_cast<char *>(a);
            }
            const int cols = p.head_dim;
            const bool any_none = __any_sync(0xffffffffu, none);
            const float2 inv2 = make_float2(inv, inv);
            // 32 columns in registers: scaled, and to the rows
            auto put = [&](uint32_t (&o)[32], int d) {
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const float2 v = PR::mul(make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), inv2);
                    o[i] = __float_as_uint(v.x);
                    o[i + 1] = __float_as_uint(v.y);
                }
                if (any_none) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = none ? 0u : o[i];
                }
                uint4 ck[4];
                if (parts) {  // fp32: two blocks of 16 values
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int i = 16 * hh + 4 * k;
                            ck[k] = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                        }
                        transpose4(ck, lane);
                        const int at = d + 16 * hh + (lane & 3) * 4;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (rows4[k] && at < cols) *reinterpret_cast<uint4 *>(rows4[k] + at * 4) = ck[k];
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t pk[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            pk[e] = pack_pair<T>(make_float2(__uint_as_float(o[8 * k + 2 * e]), __uint_as_float(o[8 * k + 2 * e + 1])));
                        ck[k] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    }
                    transpose4(ck, lane);
                    const int at = d + (lane & 3) * 8;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (!rows4[k] || at >= cols) continue;
                        if (p.out_vec)
                            *reinterpret_cast<uint4 *>(rows4[k] + at * 2) = ck[k];
                        else
                            store_halves(reinterpret_cast<uint16_t *>(rows4[k]) + at, ck[k]);
                    }
                }
            };
            if (!(ok = o_ready())) break;
            // (rolled: unrolled further, the code's fetches took longer than the work)
#pragma unroll 1
            for (int d = 0; d < cols; d += 64) {
                uint32_t oa[32], ob[32];
                __syncwarp();
                tmem_ld32(to + d, oa);
                tmem_ld32(to + d + 32, ob);
                tmem_wait_ld();
                put(oa, d);
                put(ob, d + 32);
            }
            // (o is read before the next item's first product, which waits for
            // this warp's next p)
            tc_before_sync();
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
    if constexpr (CL) {
        __syncwarp();
        cluster_sync();
        join_cluster<T, DP>(p, items[0], join_at, join_lse);
        __syncwarp();
        cluster_sync();  // no CTA ends while another reads its rows
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
    const int q0 = min(max(p.cu_q[b], 0), T_);
    const int nq = min(max(p.cu_q[b + 1], q0), T_) - q0;
    if (tok >= nq) return;
    const int kv = kv_length(p, p.kv_lens[b]);
    // a row tile whose keys one split held has written its rows itself
    const int per = p.nq * p.tile_toks, tile_end = min((tok / per + 1) * per, min(nq, p.max_q));
    const int lim = keys_seen(p, kv, nq, tile_end);
    if (lim > 0 && lim <= p.chunk) return;
    const int64_t seen = keys_seen(p, kv, nq, tok + 1);
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
    bool cluster;  // the splits of a row are a cluster
    size_t workspace;
};

// held[s]: clusters of s CTAs that the device holds at once.
static AttnCut attn_cut(const paged_attn_call_t &c, int sms, const int32_t *held) {
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
    k.cluster = false;
    // CTAs for each row tile, a split being worth two key tiles at least
    const int64_t want = ctas < slots ? std::min(slots / ctas, tiles / 2) : 1;
    if (want > 1) {
        int64_t per_split = (tiles + want - 1) / want;
        // A cluster joins its splits itself; otherwise a second kernel does,
        // which takes as long as a few key tiles. A cluster lies in one part of
        // the device (which has parts of unequal sizes: 14 clusters of 16, not 16);
        // its size is such that they all fit at once (two sequences of 8192
        // keys, 8 key heads: 16 clusters of 16, two of them late, 27.4 us; of 13,
        // 17.5; five sequences: 40 clusters of 7, of which 38 fit, 50.7, of 6 32.2).
        int64_t size = kClusterMost;
        while (size > 1 && held[size] < ctas) --size;
        const int64_t per_cluster = (tiles + size - 1) / size;
        k.cluster = k.nq == 1 && size > 1 && per_cluster - per_split <= kJoinTiles;
        if (k.cluster && per_split < per_cluster) per_split = per_cluster;
        k.splits = (int)((tiles + per_split - 1) / per_split);
        k.chunk = (int)(per_split * kKeyTile);
        if (k.splits < 2) k.cluster = false;
    } else if (k.nq == 1 && ctas < 4 * slots && tiles >= 2 * kDecodeChunk) {
        // Up to a few items a CTA: shorter ones let the CTAs end together where
        // the lengths differ (lengths of 964 to 8192 keys, 8 key heads: 24
        // sequences 119 -> 87 us, 32: 122 -> 105, 64: 219 -> 195; 8192 each:
        // 129 -> 132, 161 -> 176, 300 -> 304). Rows by the hundred lose more
        // with their partial results (chunks of 512 over 8192: 124 -> 147 us in
        // two).
        // max_kv is a bound that the lengths may be far below (one captured call
        // for every length): the number of items is held, and with it the
        // workspace and the empty items, each of which a CTA asks for and drops.
        // Beyond 32 a CTA the items get longer instead. (64 sequences of 964 to
        // 8192 keys, 193 us: called with max_kv 2^17 219 us, as without the limit;
        // with 2^20 225 us and 20 MB, against 532 us and 541 MB.)
        const int64_t most = kDecodeItems * slots / ctas;
        const int64_t per_split = std::max((int64_t)kDecodeChunk, (tiles + most - 1) / most);
        k.splits = (int)((tiles + per_split - 1) / per_split);
        k.chunk = (int)(per_split * kKeyTile);
    }
    k.workspace = 0;
    if (k.splits > 1 && !k.cluster) {
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
    if (c.max_kv > 0x7fffffff - 2 * kKeyTile) return RMSNORM_ERR_UNSUPPORTED;  // a tile's keys are counted in 32 bits
    return RMSNORM_SUCCESS;
}

template <typename T, int DP, int NQ, bool CL>
static int launch_attn(const AttnParams &p, const CUtensorMap (&maps)[3], unsigned grid, cudaStream_t stream) {
    using S = AttnShape<DP, NQ>;
    auto *kernel = paged_attn<T, DP, NQ, CL>;
    const int e = allow_staged_smem(reinterpret_cast<const void *>(kernel));
    if (e != 0) return e;
    if (CL && p.splits > 8) {
        const cudaError_t ce = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (ce != cudaSuccess) {
            (void)cudaGetLastError();
            return (int)ce;
        }
    }
    LaunchCfg lc(grid, S::kThreads, S::kSmem, stream, CL ? (unsigned)p.splits : 0);
    return (int)cudaLaunchKernelEx(&lc.cfg, kernel, p, maps[0], maps[1], maps[2]);
}

// attn_cut's `held` for the current device, asked once per device and head
// size: [kClusterMost + 1] counts; 0 where the device has no room or no answer,
// and the join's kernel serves. The runtime takes any kernel with tensor memory
// for one CTA an SM (7 clusters of 16 on a GB300, where 14 run at once, as CTAs
// that noted their start and end showed), so it is asked about one without:
// never launched, with the threads, shared memory and bound on registers of
// paged_attn<T, DP, 1, true>, whose 256 columns are half an SM's.
__global__ void __launch_bounds__(256, 2) attn_cluster_room() {}

template <int DP> static const int32_t *clusters_held(int dev, int sms) {
    using S = AttnShape<DP, 1>;
    static_assert(S::kThreads == 256 && S::kCols <= 256, "two CTAs an SM");
    static std::mutex mu;
    static int32_t held[64][kClusterMost + 1];
    static bool asked[64];
    std::lock_guard<std::mutex> lk(mu);
    if (!asked[dev]) {
        auto *kernel = attn_cluster_room;
        bool ok = allow_staged_smem(reinterpret_cast<const void *>(kernel)) == 0;
        const bool wide = ok && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
        for (int size = 2; ok && size <= (wide ? kClusterMost : 8); ++size) {
            LaunchCfg lc((unsigned)(size * sms), S::kThreads, S::kSmem, nullptr, (unsigned)size, false);
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, kernel, &lc.cfg) == cudaSuccess) held[dev][size] = n;
        }
        (void)cudaGetLastError();
        asked[dev] = true;
    }
    return held[dev];
}

// The cut of a call on the current device; a cudaError_t.
static int cut_here(const paged_attn_call_t &c, AttnCut &cut, int **status) {
    int dev = 0, sms = 0;
    const int e = current_device(&sms, status, &dev);
    if (e == 0) cut = attn_cut(c, sms, c.head_dim > 64 ? clusters_held<128>(dev, sms) : clusters_held<64>(dev, sms));
    return e;
}

template <typename T, int DP>
static int launch_attn_d(const AttnCut &k, const AttnParams &p, const CUtensorMap (&maps)[3], unsigned grid, cudaStream_t s) {
    if (k.nq == 2) return launch_attn<T, DP, 2, false>(p, maps, grid, s);
    return k.cluster ? launch_attn<T, DP, 1, true>(p, maps, grid, s) : launch_attn<T, DP, 1, false>(p, maps, grid, s);
}

template <typename T>
static int launch_attn_t(const AttnCut &k, const AttnParams &p, const CUtensorMap (&maps)[3], unsigned grid, cudaStream_t s) {
    return p.head_dim > 64 ? launch_attn_d<T, 128>(k, p, maps, grid, s) : launch_attn_d<T, 64>(k, p, maps, grid, s);
}

static rmsnorm_status_t attn_impl(const paged_attn_call_t &c, cudaStream_t stream) {
    rmsnorm_status_t st = attn_sizes(c);
    if (st != RMSNORM_SUCCESS) return st;
    const float log2_scale = c.scale * 1.44269504088896340736f;
    if (!std::isfinite(log2_scale) || !(log2_scale > 0.f)) return RMSNORM_ERR_INVALID_ARG;
    const paged_cache_t &pc = c.cache;
    if (pc.page_size < 1 || pc.pages < 0 || pc.pages > 0x7ffffffeLL) return RMSNORM_ERR_INVALID_ARG;
    if (pc.page_size % 8 != 0) return RMSNORM_ERR_UNSUPPORTED;
    if (c.workspace && !on(c.workspace, 16)) return RMSNORM_ERR_WORKSPACE;
    if (c.tokens == 0 || c.batch == 0 || c.max_q == 0) return RMSNORM_SUCCESS;
    if (!c.q || !c.out || !on(c.q, 2) || !on(c.out, 2) || !on(c.lse, 4) || !c.kv_lens || !c.cu_q ||
        !on(c.block_table, 4) || !on(c.kv_lens, 4) || !on(c.cu_q, 4) || !apart(c.out_token, c.tokens) ||
        !apart(c.out_head, c.q_heads))
        return RMSNORM_ERR_INVALID_ARG;
    // without a page every sequence is empty; the kernel then reads no table
    const bool empty = pc.pages == 0 || c.table_width == 0 || c.max_kv == 0;
    if (!empty && (!pc.k || !pc.v || !c.block_table)) return RMSNORM_ERR_INVALID_ARG;

    auto legal = [&](const void *base, int64_t page, int64_t slot, int64_t head) {
        return on(base, 16) && tile_stride(page, pc.pages) && tile_stride(slot, pc.page_size) && tile_stride(head, pc.heads);
    };
    if (!empty && (!legal(pc.k, pc.k_page, pc.k_slot, pc.k_head) || !legal(pc.v, pc.v_page, pc.v_slot, pc.v_head)))
        return RMSNORM_ERR_UNSUPPORTED;

    paged_attn_call_t cc = c;
    if (empty) cc.max_kv = 0;
    AttnCut cut;
    int *status = nullptr;
    const int e = cut_here(cc, cut, &status);
    if (e != 0) return head_cuda_fail(e);

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
    p.c = log2_scale;
    p.batch = c.batch;
    p.width = empty ? 0 : c.table_width;
    p.heads = c.q_heads;
    p.group = c.q_heads / pc.heads;
    p.head_dim = c.head_dim;
    p.pages = (int)pc.pages;
    p.page_size = pc.page_size;
    while ((1 << p.box_log2) < p.box_rows) ++p.box_log2;
    p.by_heads = Divisor::of(pc.heads);
    p.by_batch = Divisor::of(c.batch);
    p.by_splits = Divisor::of(cut.splits);
    p.by_page = Divisor::of(pc.page_size);
    p.by_group = Divisor::of(c.q_heads / pc.heads);
    p.max_q = c.max_q;
    p.max_kv = cc.max_kv;
    p.causal = c.causal != 0;
    p.q_tiles = cut.q_tiles;
    p.splits = cut.splits;
    p.chunk = cut.chunk;
    p.tile_toks = cut.tile_toks;
    p.nq = cut.nq;
    p.by_seq = !cut.cluster && c.batch > 1 && c.batch <= 32 && cc.max_kv / 2 >= c.max_q;
    // (a group's heads share a box: their stride counts even for one key head)
    if (!empty && on(c.q, 16) && tile_stride(c.q_head, c.q_heads) && tile_stride(c.q_token, c.tokens))
        p.q_tma = tile_map(&maps[0], c.dtype, c.q, c.head_dim, {p.group, pc.heads, c.tokens},
                           {c.q_head, c.q_head * p.group, c.q_token}, p.group, p.tile_toks);
    const int pieces = kKeyTile / p.box_rows * (c.head_dim > 64 ? 2 : 1);
    p.copiers = pieces > (cut.nq == 1 ? 16 : 8) ? 3 : 1;
    p.q_vec = on(c.q, 16) && p.q_token % 16 == 0 && p.q_head % 16 == 0;
    p.out_vec = on(c.out, 16) && p.out_token % 16 == 0 && p.out_head % 16 == 0;

    const int64_t grid = (int64_t)c.batch * pc.heads * cut.q_tiles * cut.splits;
    const int64_t join = ((int64_t)c.batch * c.max_q * c.q_heads + 3) / 4;
    int le = 0;
    const bool joins = cut.splits > 1 && !cut.cluster;
    if (grid > 0x7fffffffLL || (joins && join > 0x7fffffffLL)) {
        st = RMSNORM_ERR_UNSUPPORTED;
    } else {
        le = c.dtype == RMSNORM_BF16 ? launch_attn_t<__nv_bfloat16>(cut, p, maps, (unsigned)grid, stream)
                                     : launch_attn_t<__half>(cut, p, maps, (unsigned)grid, stream);
        if (le == 0 && joins) {
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
    AttnCut cut;
    return cut_here(*call, cut, nullptr) == 0 ? cut.workspace : 0;
}

extern "C" rmsnorm_status_t paged_attn_plan_query(const paged_attn_call_t *call, int32_t num_sms, const int32_t *clusters,
                                                  paged_attn_plan_t *plan) {
    if (!call || !plan || (num_sms > 0 && !clusters)) return RMSNORM_ERR_INVALID_ARG;
    const rmsnorm_status_t st = attn_sizes(*call);
    if (st != RMSNORM_SUCCESS) return st;
    if (call->tokens == 0 || call->batch == 0 || call->max_q == 0) return RMSNORM_ERR_INVALID_ARG;
    AttnCut cut;
    if (num_sms > 0) {
        cut = attn_cut(*call, num_sms, clusters);
    } else {
        const int e = cut_here(*call, cut, nullptr);
        if (e != 0) return head_cuda_fail(e);
    }
    *plan = paged_attn_plan_t{cut.nq, cut.tile_toks, cut.q_tiles, cut.splits, cut.chunk, cut.cluster ? 1 : 0,
                              (int64_t)cut.workspace};
    return RMSNORM_SUCCESS;
}
