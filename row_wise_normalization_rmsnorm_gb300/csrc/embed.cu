// embed.cu -- the gradient of embedding rows:  dtable_v = scale sum_{t: id_t = v} dh_t.
//
// Tokens are sorted by id, stably, so that a row's gradient is one run of
// tokens in their order: its sum has one order whatever the launch does, with
// no atomics on values. Runs are of very unlike lengths (a text's tokens
// follow a power law), so the sorted tokens are cut into pieces of 32 (few
// values: 8) that a team each sums. A run inside a piece goes to its row at once; what a piece
// has of a run that goes on beyond it is joined in a second launch. A sum has a piece's tokens
// in sequence, then a quarter of its run's pieces, then the quarters.
// Rows without a token are set to zero by other CTAs of the first launch.
//
// Bytes: T N of dh read and V N of dtable written, once each; the sort moves
// 8 bytes a token in shared memory.
#include "embed.cuh"

#include "groupnorm_kernels.cuh"

namespace rmsn {

// -------------------------------------------------------------------- sort --
// Least significant digit first, up to 9 bits a pass (ids below 2^18: two
// passes). A warp ranks 32 tokens at a time among equal digits (match), its
// own counts giving the ranks before; the warps', the CTAs' and the digits'
// counts are then added up.

__device__ __forceinline__ uint32_t key_of(const SortParams &p, int t) {
    const int64_t id = p.id_bytes == 8 ? static_cast<const int64_t *>(p.ids)[t] : (int64_t) static_cast<const int32_t *>(p.ids)[t];
    return id >= 0 && id < p.rows ? (uint32_t)id : (uint32_t)p.rows;
}

struct SortShared {
    uint16_t warp[kSortThreads / 32][kSortBins];  // a warp's tokens of a digit, then those of the warps before it
    uint32_t total[kSortBins];                    // this CTA's
    uint32_t base[kSortBins];                     // where this CTA's tokens of a digit begin
    uint32_t scan[kSortThreads / 32];
};

// The places among equal digits of this thread's tokens (n tokens of a CTA,
// `per` rounds of 32 for each warp, a warp's tokens neighbours), and the
// CTA's totals.
template <int PER, class Key>
__device__ __forceinline__ void rank_tokens(SortShared &s, int n, int per, int shift, int bits, Key &&key, uint32_t (&rank)[PER]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bins = 1 << bits;
    for (int d = lane; d < bins; d += 32) s.warp[warp][d] = 0;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        if (r < per) {
            const int i = (warp * per + r) * 32 + lane;
            const bool in = i < n;
            const uint32_t d = in ? (key(r) >> shift) & (uint32_t)(bins - 1) : (uint32_t)bins;  // a digit that none has
            const uint32_t same = __match_any_sync(0xffffffffu, d);
            const uint32_t before = __popc(same & ((1u << lane) - 1u));
            const uint32_t have = in ? s.warp[warp][d] : 0u;
            rank[r] = have + before;
            __syncwarp();
            if (in && before == 0) s.warp[warp][d] = (uint16_t)(have + __popc(same));
            __syncwarp();
        }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < bins; d += kSortThreads) {
        uint32_t t = 0;
        for (int w = 0; w < kSortThreads / 32; ++w) {
            const uint32_t c = s.warp[w][d];
            s.warp[w][d] = (uint16_t)t;
            t += c;
        }
        s.total[d] = t;
    }
    __syncthreads();
}

// Exclusive sums of up to kSortBins values, one a thread; all threads call it.
__device__ __forceinline__ uint32_t bins_before(SortShared &s, uint32_t v) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s.scan[warp] = x;
    __syncthreads();
    if (warp == 0) {
        uint32_t w = s.scan[lane];
        uint32_t z = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, z, o);
            if (lane >= o) z += y;
        }
        s.scan[lane] = z - w;
    }
    __syncthreads();
    return x - v + s.scan[warp];
}

__device__ __forceinline__ uint32_t cluster_address(const void *local, uint32_t cta) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(local)), "r"(cta));
    return r;
}
__device__ __forceinline__ uint32_t cluster_ctas() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t ld_remote(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void st_remote2(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}

// E values of a row of the table, as up to 16 bytes an access.
template <typename TO, int E> __device__ __forceinline__ void clear_row(void *dtable, int64_t row, int N, int c) {
    constexpr int S = E * (int)sizeof(TO) > 16 ? 16 / (int)sizeof(TO) : E;
    float zero[S];
    fill_v(0.f, zero);
    Vals<TO, S> o;
    o.set(zero);
#pragma unroll
    for (int k = 0; k < E; k += S) o.store(static_cast<TO *>(dtable) + row * N + (int64_t)c * E + k);
}

// The rows without a token, by the CTAs beside the sorting cluster: each
// marks the ids of its share of the rows in shared memory, then clears the
// others. The sort keeps 8 SMs for 15 us, and memory would be idle; as many
// rows are cleared here as memory takes in that time (it writes 3.9 TB/s at
// most, reads and writes 6.7 together), the others beside the sums.
template <typename TO, int E> __device__ __forceinline__ void clear_rows(const SortParams &p, uint32_t *marks, int cta, int ctas) {
    const int64_t v0 = p.early * cta / ctas, v1 = p.early * (cta + 1) / ctas;
    const int C = p.N / E, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t lo = v0; lo < v1; lo += (int64_t)kClearWords * 32) {
        const int n = (int)min((int64_t)kClearWords * 32, v1 - lo);
        for (int i = threadIdx.x; i < (n + 31) / 32; i += kSortThreads) marks[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int t = threadIdx.x; t < p.T; t += kSortThreads) {
            const int64_t k = (int64_t)key_of(p, t) - lo;
            // (a look first: the same few ids come over and over)
            if (k >= 0 && k < n && !(*(volatile uint32_t *)&marks[k >> 5] >> (k & 31) & 1u)) atomicOr(&marks[k >> 5], 1u << (k & 31));
        }
        __syncthreads();
        for (int r = warp; r < n; r += kSortThreads / 32)
            if (!(marks[r >> 5] >> (r & 31) & 1u))
                for (int c = lane; c < C; c += 32) clear_row<TO, E>(p.dtable, lo + r, p.N, c);
        __syncthreads();
    }
}

// Up to kSortCluster kSortTile tokens: one cluster, (id, token) pairs in its
// shared memory between the passes, each CTA an equal share of the places.
// smem: SortShared, then two buffers of `share` pairs.
constexpr int kSortPer = kSortTile / kSortThreads;
template <typename TO, int E> __global__ void __launch_bounds__(kSortThreads) embed_sort(const SortParams p, int share) {
    extern __shared__ __align__(16) uint8_t raw[];
    SortShared &s = *reinterpret_cast<SortShared *>(raw);
    uint2 *buf[2] = {reinterpret_cast<uint2 *>(raw + sizeof(SortShared)), reinterpret_cast<uint2 *>(raw + sizeof(SortShared)) + share};
    pdl_wait();
    pdl_trigger();
    const int ctas = (int)cluster_ctas(), rank = (int)cluster_ctarank();
    if ((int)blockIdx.x >= ctas) {
        clear_rows<TO, E>(p, reinterpret_cast<uint32_t *>(raw + sizeof(SortShared)), (int)blockIdx.x - ctas, (int)gridDim.x - ctas);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = max(0, min(share, p.T - rank * share));
    const int per = (share + kSortThreads - 1) / kSortThreads;
    for (int i = rank * kSortThreads + threadIdx.x; i < p.words; i += ctas * kSortThreads) p.present[i] = 0;
    if (rank == 0 && threadIdx.x == 0) p.open[0] = 0;
    uint32_t key[kSortPer], val[kSortPer], place[kSortPer];
#pragma unroll
    for (int r = 0; r < kSortPer; ++r) {
        const int i = (warp * per + r) * 32 + lane;
        val[r] = (uint32_t)(rank * share + i);
        key[r] = r < per && i < n ? key_of(p, rank * share + i) : 0u;
    }
    for (int pass = 0; pass < p.passes; ++pass) {
        if (pass > 0) {
            const uint2 *b = buf[pass & 1];
#pragma unroll
            for (int r = 0; r < kSortPer; ++r) {
                const int i = (warp * per + r) * 32 + lane;
                if (r < per && i < n) {
                    key[r] = b[i].x;
                    val[r] = b[i].y;
                }
            }
        }
        const int shift = pass * p.bits;
        rank_tokens<kSortPer>(s, n, per, shift, p.bits, [&](int r) { return key[r]; }, place);
        cluster_sync();  // the CTAs' totals (and, before the first pass, the cleared bits) are there
        uint32_t all = 0, before = 0;
        if ((int)threadIdx.x < (1 << p.bits))
            for (int c = 0; c < ctas; ++c) {
                const uint32_t t = ld_remote(cluster_address(&s.total[threadIdx.x], (uint32_t)c));
                all += t;
                if (c < rank) before += t;
            }
        const uint32_t lower = bins_before(s, all);
        if ((int)threadIdx.x < (1 << p.bits)) s.base[threadIdx.x] = lower + before;
        __syncthreads();
        const bool last = pass == p.passes - 1;
#pragma unroll
        for (int r = 0; r < kSortPer; ++r) {
            const int i = (warp * per + r) * 32 + lane;
            if (r < per && i < n) {
                const uint32_t d = (key[r] >> shift) & ((1u << p.bits) - 1u);
                const uint32_t to = s.base[d] + s.warp[warp][d] + place[r];
                if (last) {
                    p.keys[to] = key[r];
                    p.vals[to] = val[r];
                } else {
                    const uint32_t cta = to / (uint32_t)share;
                    st_remote2(cluster_address(&buf[(pass + 1) & 1][to - cta * share], cta), key[r], val[r]);
                }
                if (pass == 0 && key[r] < (uint32_t)p.rows) atomicOr(&p.present[key[r] >> 5], 1u << (key[r] & 31u));
            }
        }
        cluster_sync();  // pairs have arrived, and nobody reads these totals any more
    }
}

// More tokens: a pass is three launches over tiles of kSortTile tokens.
__device__ __forceinline__ void tile_tokens(const SortParams &p, uint32_t (&key)[kSortPer], uint32_t (&val)[kSortPer], int n) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int r = 0; r < kSortPer; ++r) {
        const int i = (warp * kSortPer + r) * 32 + lane, t = blockIdx.x * kSortTile + i;
        key[r] = i < n ? (p.keys_in ? p.keys_in[t] : key_of(p, t)) : 0u;
        val[r] = i < n ? (p.keys_in ? p.vals_in[t] : (uint32_t)t) : 0u;
    }
}
__global__ void __launch_bounds__(kSortThreads) embed_sort_count(const SortParams p) {
    extern __shared__ __align__(16) uint8_t raw[];
    SortShared &s = *reinterpret_cast<SortShared *>(raw);
    pdl_wait();
    pdl_trigger();
    uint32_t key[kSortPer], val[kSortPer], place[kSortPer];
    const int n = min(kSortTile, p.T - (int)blockIdx.x * kSortTile);
    tile_tokens(p, key, val, n);
    rank_tokens<kSortPer>(s, n, kSortPer, p.shift, p.bits, [&](int r) { return key[r]; }, place);
    for (int d = threadIdx.x; d < (1 << p.bits); d += kSortThreads) p.counts[(int64_t)d * p.tiles + blockIdx.x] = s.total[d];
}
// A CTA a digit: its counts become the tokens of that digit in the tiles before.
__global__ void __launch_bounds__(kSortThreads) embed_sort_scan(const SortParams p) {
    __shared__ SortShared s;
    pdl_wait();
    pdl_trigger();
    uint32_t *c = p.counts + (int64_t)blockIdx.x * p.tiles;
    uint32_t sum = 0;
    for (int t0 = 0; t0 < p.tiles; t0 += kSortThreads) {
        const int t = t0 + threadIdx.x;
        const uint32_t v = t < p.tiles ? c[t] : 0u;
        const uint32_t before = bins_before(s, v);
        if (t < p.tiles) c[t] = sum + before;
        if (threadIdx.x == kSortThreads - 1) s.base[0] = before + v;
        __syncthreads();
        sum += s.base[0];
        __syncthreads();
    }
    if (threadIdx.x == 0) p.counts[(int64_t)kSortBins * p.tiles + blockIdx.x] = sum;
}
__global__ void __launch_bounds__(kSortThreads) embed_sort_move(const SortParams p) {
    extern __shared__ __align__(16) uint8_t raw[];
    SortShared &s = *reinterpret_cast<SortShared *>(raw);
    pdl_wait();
    pdl_trigger();
    uint32_t key[kSortPer], val[kSortPer], place[kSortPer];
    const int n = min(kSortTile, p.T - (int)blockIdx.x * kSortTile);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    tile_tokens(p, key, val, n);
    rank_tokens<kSortPer>(s, n, kSortPer, p.shift, p.bits, [&](int r) { return key[r]; }, place);
    const bool mine = (int)threadIdx.x < (1 << p.bits);
    const uint32_t lower = bins_before(s, mine ? p.counts[(int64_t)kSortBins * p.tiles + threadIdx.x] : 0u);
    if (mine) s.base[threadIdx.x] = lower + p.counts[(int64_t)threadIdx.x * p.tiles + blockIdx.x];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSortPer; ++r) {
        const int i = (warp * kSortPer + r) * 32 + lane;
        if (i < n) {
            const uint32_t d = (key[r] >> p.shift) & ((1u << p.bits) - 1u);
            const uint32_t to = s.base[d] + s.warp[warp][d] + place[r];
            p.keys[to] = key[r];
            p.vals[to] = val[r];
            // (the bits were cleared before the first pass)
            if (p.shift == 0 && key[r] < (uint32_t)p.rows) atomicOr(&p.present[key[r] >> 5], 1u << (key[r] & 31u));
        }
    }
}

// --------------------------------------------------------------------- sum --

// scale times the sum of a row's tokens, to its row of the table (added to
// what is there, where the caller accumulates; one rounding either way).
template <typename TO, int E>
__device__ __forceinline__ void give_row(const EmbedSumParams &p, uint32_t row, int c, const float (&sum)[E]) {
    TO *to = static_cast<TO *>(p.dtable) + (int64_t)row * p.N + (int64_t)c * E;
    float v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = sum[i] * p.scale;
    constexpr int S = E * (int)sizeof(TO) > 16 ? 16 / (int)sizeof(TO) : E;  // values of one access
#pragma unroll
    for (int k = 0; k < E; k += S) {
        Vals<TO, S> o;
        float w[S];
        if (p.accumulate) {
            o.load(to + k);
            o.get(w);
#pragma unroll
            for (int i = 0; i < S; ++i) w[i] = fmaf(sum[k + i], p.scale, w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < S; ++i) w[i] = v[k + i];
        }
        o.set(w);
        o.store(to + k);
    }
}
template <int E> __device__ __forceinline__ float *part_at(const EmbedSumParams &p, int piece, int last, int c) {
    return p.parts + ((int64_t)piece * 2 + last) * p.N + (int64_t)c * E;
}

constexpr int kSumBatch = 8;  // a team's tokens under way at once

// CTAs 0 .. sum_ctas - 1: a team of `team` threads a piece and a slice of
// `team` chunks of the row. The CTAs behind them: 32 rows of the table and a
// slice each, of which those without a token are set to zero.
template <typename T, typename TO, int E>
__global__ void __launch_bounds__(256) embed_sum(const EmbedSumParams p) {
    __shared__ uint32_t key[256 / 8][kEmbedPiece + 2], val[256 / 8][kEmbedPiece];
    pdl_wait();
    pdl_trigger();
    const int C = p.N / E;
    if ((int)blockIdx.x >= p.sum_ctas) {
        const int64_t item = (int64_t)blockIdx.x - p.sum_ctas;
        const int64_t r0 = p.early + item / p.slices * 32;
        const uint32_t there = p.present[r0 >> 5];
        const int teams = 256 / p.team;
        const int c = (int)(item % p.slices) * p.team + (int)threadIdx.x % p.team;
        if (c < C)
            for (int r = threadIdx.x / p.team; r < 32 && r0 + r < p.rows; r += teams)
                if (!(there >> r & 1u)) clear_row<TO, E>(p.dtable, r0 + r, p.N, c);
        return;
    }
    const int team = threadIdx.x / p.team, t = threadIdx.x % p.team, teams = 256 / p.team;
    const int64_t item = (int64_t)blockIdx.x * teams + team;
    const int piece = (int)(item / p.slices);
    const int c = (int)(item - (int64_t)piece * p.slices) * p.team + t;
    const int at = piece * p.piece;
    const int n = piece < p.pieces ? min(p.piece, p.T - at) : 0;
    // the piece's ids with a neighbour on either side, and its tokens
    for (int i = t; i < p.piece + 2; i += p.team) {
        const int g = at + i - 1;
        key[team][i] = n > 0 && i <= n + 1 && g >= 0 && g < p.T ? p.keys[g] : 0xffffffffu;  // of no row
        if (i < n) val[team][i] = p.vals[at + i];
    }
    __syncthreads();
    if (n == 0 || c >= C) return;
    const T *dh = static_cast<const T *>(p.dh) + (int64_t)c * E;
    float sum[E];
#pragma unroll
    for (int i = 0; i < E; ++i) sum[i] = 0.f;
    bool whole = key[team][0] != key[team][1];  // the run that is being summed began in this piece
    for (int k = 0; k < n; k += kSumBatch) {
        Vals<T, E> v[kSumBatch];
#pragma unroll
        for (int q = 0; q < kSumBatch; ++q)
            if (k + q < n && key[team][k + q + 1] < (uint32_t)p.rows) v[q].load_last(dh + (int64_t)val[team][k + q] * p.N);
#pragma unroll
        for (int q = 0; q < kSumBatch; ++q) {
            const uint32_t id = k + q < n ? key[team][k + q + 1] : 0xffffffffu;
            if (id < (uint32_t)p.rows) {
                float f[E];
                v[q].get(f);
#pragma unroll
                for (int i = 0; i < E; ++i) sum[i] += f[i];
                const bool ends = key[team][k + q + 2] != id;
                if (ends || k + q + 1 == n) {
                    if (ends && whole) {
                        give_row<TO, E>(p, id, c, sum);
                    } else {
                        float *to = part_at<E>(p, piece, whole ? 1 : 0, c);
#pragma unroll
                        for (int i = 0; i < E; ++i) to[i] = sum[i];
                        if (c == 0 && ends) p.ends[id] = (uint32_t)piece;
                        if (c == 0 && whole) {  // in any order
                            const uint32_t i = atomicAdd(p.open, 1u);
                            *reinterpret_cast<uint2 *>(p.open + 2 + 2 * i) = make_uint2((uint32_t)piece, id);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < E; ++i) sum[i] = 0.f;
                    whole = true;
                }
            }
        }
    }
}

// Runs over several pieces: the last part of the piece where the run begins,
// then the first parts of those behind it, in order. kJoinLanes lanes of
// pieces and kJoinChunks chunks a CTA; the lanes' sums are added in order.
template <typename T, typename TO, int E>
__global__ void __launch_bounds__(256) embed_join(const EmbedSumParams p) {
    __shared__ float lane_sum[kJoinLanes][kJoinChunks][E + 1];
    pdl_wait();
    pdl_trigger();
    const int C = p.N / E, slices = (C + kJoinChunks - 1) / kJoinChunks;
    const int64_t items = (int64_t)p.open[0] * slices;
    const int lane = threadIdx.x / kJoinChunks, t = threadIdx.x % kJoinChunks;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const uint2 run = *reinterpret_cast<const uint2 *>(p.open + 2 + 2 * (item / slices));
        const int first = (int)run.x, last = (int)p.ends[run.y];
        const int c = (int)(item % slices) * kJoinChunks + t;
        const int per = (last - first + kJoinLanes) / kJoinLanes, lanes = (last - first + per) / per;  // lanes with pieces
        float sum[E];
        fill_v(0.f, sum);
        if (c < C && lane < lanes) {
            const int k0 = first + lane * per, k1 = min(k0 + per, last + 1);
#pragma unroll 4
            for (int k = k0; k < k1; ++k) {
                const float *part = part_at<E>(p, k, k == first ? 1 : 0, c);
#pragma unroll
                for (int i = 0; i < E; ++i) sum[i] += part[i];
            }
        }
#pragma unroll
        for (int i = 0; i < E; ++i) lane_sum[lane][t][i] = sum[i];
        __syncthreads();
        if (lane == 0 && c < C) {
            for (int l = 1; l < lanes; ++l)
#pragma unroll
                for (int i = 0; i < E; ++i) sum[i] += lane_sum[l][t][i];
            give_row<TO, E>(p, run.y, c, sum);
        }
        __syncthreads();
    }
}

const void *sort_kernel(int which) {
    return which == 1   ? (const void *)embed_sort_count
           : which == 2 ? (const void *)embed_sort_scan
                        : (const void *)embed_sort_move;
}
size_t sort_shared() { return sizeof(SortShared); }

enum { kPickSort, kPickSum, kPickJoin };
template <typename T, typename TO, int E> static const void *embed_kernel(int which) {
    return which == kPickSort  ? (const void *)embed_sort<TO, E>
           : which == kPickSum ? (const void *)embed_sum<T, TO, E>
                               : (const void *)embed_join<T, TO, E>;
}
static const void *embed_pick(int which, int dtype, bool out32, bool wide) {
#define PICK(T, TO) (wide ? embed_kernel<T, TO, Elem<T>::E>(which) : embed_kernel<T, TO, 1>(which))
    if (dtype == 0) return PICK(float, float);
    if (dtype == 1) return out32 ? PICK(__nv_bfloat16, float) : PICK(__nv_bfloat16, __nv_bfloat16);
    return out32 ? PICK(__half, float) : PICK(__half, __half);
#undef PICK
}
const void *embed_sort_kernel(int dtype, bool out32, bool wide) { return embed_pick(kPickSort, dtype, out32, wide); }
const void *embed_sum_kernel(int dtype, bool out32, bool wide) { return embed_pick(kPickSum, dtype, out32, wide); }
const void *embed_join_kernel(int dtype, bool out32, bool wide) { return embed_pick(kPickJoin, dtype, out32, wide); }

}  // namespace rmsn
