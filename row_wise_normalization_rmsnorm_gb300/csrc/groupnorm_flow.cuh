// groupnorm_flow.cuh -- group norm of samples that no cluster holds: one launch
// of persistent CTAs that take pieces (rows of a sample) by ticket, first to
// sum them and, `lag` pieces behind the sample's last sum, to normalise them.
// By then the sample is summed, and reads and writes overlap from there on.
// Rows are read twice, and by memory both times where a sample and the lag (of
// 8 x 65536 x 256 in bf16: 33 and 58 MB, and as much of y) are more than the L2
// keeps between the two.
//
// One warp draws the tickets and keeps a ring of stages of rows under way into
// shared memory (bulk copies, whatever alignment rows have; the sample's
// statistics with them once they are joined); eight take the stages in order;
// one joins. A piece waits only for pieces with earlier tickets, and every CTA
// takes its tickets in order: the earliest ticket not yet done is the next of
// some running CTA and waits for none, so the launch makes progress however
// few of its CTAs run at once.
//
// 8 images of 65536 x 256 in bf16: 143 us, 3.75 TB/s of bytes that are needed;
// memory reads 530 MB for the 268 of x and takes 268 of y, 5.6 TB/s. The
// gradient: 267 us, 1072 MB read for 537. (Hints to the L2 that the second
// reading and the stores are not read again changed nothing.)
//
// A piece's group statistics, (mean, sum of squared deviations) or the two
// sums of the gradient, go to memory. They are joined in two steps, kFlowFan
// neighbouring pieces by the CTA that brings the last of them, then a sample's
// fans by the one that brings the last of those, in their order: the sample
// waits for two rounds of loads, however many pieces it has. (One join of all
// pieces kept the sample waiting for 25 to 90 us.)
#pragma once

#include "groupnorm_kernels.cuh"

namespace rmsn {

constexpr int kFlowThreads = 256, kFlowCtas = 2;  // that compute, of a CTA; CTAs an SM
constexpr int kFlowAll = kFlowThreads + 64;  // threads of a CTA
constexpr int kFlowStagesMost = 8;
constexpr int kFlowMail = 4;
constexpr int kFlowFan = 16;
// Polls before a wait gives up, each wait longer than those it depends on.
constexpr uint32_t kFlowStatLimit = 1u << 22;   // of a sample's statistics (with 100 ns between: some 4 s)
constexpr uint32_t kFlowEmptyLimit = 1u << 22;  // of a stage's readers (a failed poll takes 1.4 us: 6 s)
constexpr uint32_t kFlowFullLimit = 1u << 23;   // of a stage's copies
constexpr uint32_t kFlowMailLimit = 1u << 27;   // of the mailbox (with 100 ns between)

struct FlowParams {
    GnParams g;          // rows: of a piece
    int pieces, lag;     // of a sample; sum and normalise tickets of a piece lie pieces + lag pairs apart
    int stage_rows, depth;
    uint32_t offset[4], stage_bytes;  // in a stage: dy (0: x or its codes), scales, statistics; its size
    int64_t tickets;
    int fans;            // ceil(pieces / kFlowFan)
    uint32_t *state;     // [0], [1]: the next ticket (64 bits); then [B] samples joined, [B] fans joined, [B, fans] pieces summed. Zeros at the start
    float2 *part;        // [B, pieces, G]
    float2 *fan;         // [B, fans, G]
    float2 *stat;        // [B, G]: (-mean, rstd), or the negated means of u gamma and of u gamma xhat
    uint32_t stat_limit; // polls of them before the launch gives up
    int *status;
};

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t *p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_release(uint32_t *p, uint32_t v) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void flow_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kFlowThreads) : "memory"); }
// The same, and true in all computing threads where `v` is in one.
__device__ __forceinline__ bool flow_sync_any(bool v) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"((uint32_t)v), "n"(kFlowThreads)
        : "memory");
    return any != 0;
}
__device__ __forceinline__ void flow_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

struct FlowShared {
    uint64_t full[kFlowStagesMost], empty[kFlowStagesMost];
    int64_t ticket[kFlowStagesMost];  // of the stage's piece; -1: no more
    int64_t mail[kFlowMail];          // pieces that are summed; -1: no more
    uint32_t sent, taken;
};

// A ticket's piece.
struct FlowPiece {
    bool normalise, there;
    int b, rows;
    int64_t item, first;  // piece of the batch, first row of the matrix
    __device__ __forceinline__ FlowPiece(const FlowParams &p, int64_t ticket) {
        normalise = ticket & 1;
        item = (ticket >> 1) - (normalise ? p.pieces + p.lag : 0);
        there = item >= 0 && item < (int64_t)p.g.B * p.pieces;
        b = there ? (int)(item / p.pieces) : 0;
        const int64_t r0 = (item - (int64_t)b * p.pieces) * p.g.rows;
        first = (int64_t)b * p.g.S + r0;
        rows = (int)min((int64_t)p.g.rows, p.g.S - r0);
    }
};

// The copying warp's one thread. N arrays of rows of row[i] bytes.
template <int N>
__device__ __forceinline__ void flow_copies(const FlowParams &p, FlowShared &s, uint8_t *ring, const void *const (&src)[N], const uint32_t (&row)[N]) {
    unsigned long long *next = reinterpret_cast<unsigned long long *>(p.state);
    unsigned long long drawn = atomicAdd(next, 1ull);
    int stage = 0;
    uint32_t phase = 1;
    bool round = false;  // the ring has gone round once
    auto advance = [&]() {
        if (++stage == p.depth) stage = 0, phase ^= 1u, round = true;
    };
    bool stuck = false, failed = false;  // no stage came free, or a sample was not joined
    while (!stuck && !failed) {
        const int64_t ticket = (int64_t)drawn;
        if (ticket >= p.tickets) break;
        drawn = atomicAdd(next, 1ull);  // (read when this one's copies are under way)
        const FlowPiece f(p, ticket);
        if (!f.there) continue;
        for (int r = 0; r < f.rows; r += p.stage_rows, advance()) {
            if (!mbar_wait(&s.empty[stage], phase, kFlowEmptyLimit)) {
                stuck = true;
                break;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            uint8_t *to = ring + (size_t)stage * p.stage_bytes;
            const uint32_t rows = (uint32_t)min(p.stage_rows, f.rows - r);
            Cover c[N];
            uint32_t bytes = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                c[i] = cover16(static_cast<const char *>(src[i]) + (f.first + r) * row[i], rows * row[i]);
                bytes += c[i].bytes;
            }
            const bool stats = f.normalise && r == 0;
            Cover cs;
            if (stats) {
                for (uint32_t k = 0; ld_acquire(p.state + 2 + f.b) == 0;) {
                    if (++k >= p.stat_limit) {
                        failed = true;
                        break;
                    }
                    __nanosleep(100);
                }
                if (failed) break;
                asm volatile("fence.proxy.async;" ::: "memory");
                cs = cover16(p.stat + (int64_t)f.b * p.g.G, (uint32_t)p.g.G * 8u);
                bytes += cs.bytes;
            }
            s.ticket[stage] = ticket;
            mbar_arrive_expect_tx(&s.full[stage], bytes);
            if (stats) bulk_g2s(to + p.offset[3], cs.src, cs.bytes, &s.full[stage]);
#pragma unroll
            for (int i = 0; i < N; ++i) bulk_g2s(to + (i ? p.offset[i] : 0u), c[i].src, c[i].bytes, &s.full[stage]);
        }
    }
    if ((stuck || failed) && p.status) *p.status = 1;
    // No copy is under way once this CTA has ended, whoever still waits for it:
    // the last of each stage, of this round of the ring or (from `stage` on) of the one before.
    for (int i = 0; i < p.depth; ++i)
        if (i < stage || round) mbar_wait(&s.full[i], i < stage ? phase ^ 1u : phase, kFlowFullLimit);
    if (!stuck && mbar_wait(&s.empty[stage], phase, kFlowEmptyLimit)) {
        s.ticket[stage] = -1;
        flow_arrive(&s.full[stage]);
    }
}
// The stages as the computing threads take them. Where a wait gives up, or the
// later stages of a piece do not come, the whole CTA ends its work. The lanes
// of a warp decide that together, at each stage. A warp that ends goes to the
// last barrier (flow_end); the others meet it there or behind the rows of
// their next sum, whichever comes first, and both of these barriers tell all
// threads that one has failed, so that none goes on to another. No thread can
// fail between two barriers of one sum.
struct FlowStages {
    int stage;
    uint32_t phase;
    bool failed;
    // the stage's piece (-1: no more, or the wait gave up)
    __device__ __forceinline__ int64_t wait(FlowShared &s) {
        if (!failed && !mbar_wait(&s.full[stage], phase, kFlowFullLimit)) failed = true;
        failed = __any_sync(0xffffffffu, failed);
        return failed ? -1 : s.ticket[stage];
    }
    // the next stage of this piece; false: it does not come
    __device__ __forceinline__ bool more(FlowShared &s, int64_t ticket) {
        if (wait(s) != ticket) failed = true;
        return !failed;
    }
    __device__ __forceinline__ void release(const FlowParams &p, FlowShared &s) {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) flow_arrive(&s.empty[stage]);
        if (++stage == p.depth) stage = 0, phase ^= 1u;
    }
};
__device__ __forceinline__ void flow_setup(const FlowParams &p, FlowShared &s) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.depth; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], kFlowThreads / 32);
        }
        s.sent = s.taken = 0;
        mbar_init_fence();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    pdl_wait();
    pdl_trigger();
    __syncthreads();
}

// Thread 0 tells the joining warp that a piece is summed (-1: that no more
// come). False: the mailbox stayed full.
__device__ __forceinline__ bool flow_mail(FlowShared &s, int64_t item) {
    volatile FlowShared &v = s;
    for (uint32_t k = 0; v.sent - v.taken >= kFlowMail; ++k) {
        if (k >= kFlowMailLimit) return false;
        __nanosleep(100);
    }
    v.mail[v.sent % kFlowMail] = item;
    __threadfence_block();
    v.sent = v.sent + 1;
    return true;
}
// A piece is summed and its sums are stored.
__device__ __forceinline__ void flow_tell(FlowShared &s, FlowStages &at, int64_t item) {
    flow_sync();
    if (threadIdx.x == 0 && !flow_mail(s, item)) at.failed = true;
}
// The computing threads' end; `met`: they have left a sum together.
__device__ __forceinline__ void flow_end(const FlowParams &p, FlowShared &s, const FlowStages &at, bool met) {
    const bool failed = met || flow_sync_any(at.failed);
    if (threadIdx.x == 0) {
        if (failed && p.status) *p.status = 1;
        flow_mail(s, -1);
    }
}
// True in the whole warp where this was the last of `n` to count: what the
// warp (and whoever told it) stored is there for the last, and what the others
// stored for it.
__device__ __forceinline__ bool last_of(uint32_t *counter, uint32_t n) {
    __syncwarp();
    uint32_t before = 0;
    if ((threadIdx.x & 31) == 0) asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
    before = __shfl_sync(0xffffffffu, before, 0);
    __syncwarp();
    return before == n - 1;
}
// The joining warp. join(from, n, rows, last, last_rows): a group's values of n
// neighbours `from[i G]`, of `rows` rows each but for the last-th, as one;
// give(b, k, value): the sample's.
template <class Join, class Give> __device__ __forceinline__ void flow_join(const FlowParams &p, FlowShared &s, Join &&join, Give &&give) {
    const int lane = threadIdx.x & 31, G = p.g.G;
    volatile FlowShared &v = s;
    uint32_t *joined = p.state + 2, *fans_done = joined + p.g.B, *pieces_done = fans_done + p.g.B;
    // rows of a piece and of a fan, and of a sample's last ones
    const int64_t fan_rows = (int64_t)p.g.rows * kFlowFan;
    const float rows = (float)p.g.rows, last_rows = (float)(p.g.S - (int64_t)(p.pieces - 1) * p.g.rows);
    const float many = (float)fan_rows, last_many = (float)(p.g.S - (int64_t)(p.fans - 1) * fan_rows);
    for (uint32_t n = 0;; ++n) {
        uint32_t k = 0;
        while (v.sent == n && ++k < kFlowMailLimit) __nanosleep(100);
        if (!__any_sync(0xffffffffu, v.sent != n)) {
            if (lane == 0 && p.status) *p.status = 1;
            return;
        }
        __threadfence_block();
        const int64_t item = v.mail[n % kFlowMail];
        __syncwarp();
        if (lane == 0) v.taken = n + 1;
        if (item < 0) return;
        const int b = (int)(item / p.pieces), fan = (int)(item - (int64_t)b * p.pieces) / kFlowFan;
        const int i0 = fan * kFlowFan, ni = min(kFlowFan, p.pieces - i0);
        const int64_t at = (int64_t)b * p.fans + fan;
        if (!last_of(pieces_done + at, (uint32_t)ni)) continue;
        for (int g = lane; g < G; g += 32)
            p.fan[at * G + g] = join(p.part + ((int64_t)b * p.pieces + i0) * G + g, ni, rows, p.pieces - 1 - i0, last_rows);
        if (!last_of(fans_done + b, (uint32_t)p.fans)) continue;
        for (int g = lane; g < G; g += 32)
            give(b, g, join(p.fan + (int64_t)b * p.fans * G + g, p.fans, many, p.fans - 1, last_many));
        __syncwarp();
        if (lane == 0) st_release(joined + b, 1u);
    }
}

template <typename T, int E, int ACT, bool KEEP>
__global__ void __launch_bounds__(kFlowAll, kFlowCtas) gn_fwd_flow(const FlowParams p) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(8) FlowShared fs;
    float *lane_mean = reinterpret_cast<float *>(ring + (size_t)p.depth * p.stage_bytes), *lane_m2 = lane_mean + kFlowThreads * E;
    float2 *acc = reinterpret_cast<float2 *>(lane_m2 + kFlowThreads * E);  // [G]: groups over several tiles; then the statistics
    const GnParams &g = p.g;
    flow_setup(p, fs);
    const uint32_t pitch = (uint32_t)g.C * sizeof(T);
    if (threadIdx.x >= kFlowThreads) {
        if (threadIdx.x == kFlowThreads) {
            const void *const src[1] = {g.x};
            const uint32_t row[1] = {pitch};
            flow_copies<1>(p, fs, ring, src, row);
        } else if (threadIdx.x >= kFlowThreads + 32) {
            // about the first one's mean, kFlowFan loads under way; `last` stands for fewer rows than the others
            auto join = [&](const float2 *from, int n, float rows, int last, float last_rows) {
                float ref = 0.f, s1 = 0.f, s2 = 0.f;
                const float each = rows * (float)g.cg, final = last_rows * (float)g.cg;
                for (int i0 = 0; i0 < n; i0 += kFlowFan) {
                    float2 v[kFlowFan];
#pragma unroll
                    for (int i = 0; i < kFlowFan; ++i) v[i] = __ldcg(from + min(i0 + i, n - 1) * g.G);
                    if (i0 == 0) ref = v[0].x;
#pragma unroll
                    for (int i = 0; i < kFlowFan; ++i) {
                        const float d = v[i].x - ref, nd = (i0 + i == last ? final : each) * d;
                        if (i0 + i < n) {
                            s1 += nd;
                            s2 += fmaf(nd, d, v[i].y);
                        }
                    }
                }
                const float m = s1 / (last < n ? each * (float)(n - 1) + final : each * (float)n);
                return make_float2(ref + m, at_least_0(s2 - s1 * m));
            };
            flow_join(p, fs, join, [&](int b, int k, float2 v) {
                const float r = 1.f / sqrtf(v.y / ((float)g.S * (float)g.cg) + g.eps);
                p.stat[(int64_t)b * g.G + k] = make_float2(-v.x, r);
                g.mean[(int64_t)b * g.G + k] = v.x;
                g.rstd[(int64_t)b * g.G + k] = r;
            });
        }
        return;
    }
    const int CC = g.C / E;
    const Cut cut(CC, kFlowThreads);
    const uint32_t ring0 = smem_u32(ring);
    FlowStages at{0, 0u, false};
    bool met = false;
    for (int64_t ticket; (ticket = at.wait(fs)) >= 0;) {
        const FlowPiece f(p, ticket);
        if (!f.normalise) {
            // (pieces of several stages where a row is one tile: the host's rule)
            for (int t0 = 0; t0 < CC; t0 += cut.cols) {
                const int cc = t0 + cut.col;
                const bool in = cut.in && cc < CC;
                float K[E], s1[E], s2[E];
                fill_v(0.f, K);
                fill_v(0.f, s1);
                fill_v(0.f, s2);
                int n = 0;
                for (int r0 = 0; r0 < f.rows; r0 += p.stage_rows) {
                    if (r0 > 0 && !at.more(fs, ticket)) break;
                    const uint32_t rows = ring0 + (uint32_t)at.stage * p.stage_bytes + addr_mod16(static_cast<const char *>(g.x) + (f.first + r0) * pitch);
                    const int more = in ? rows_of_lane(min(p.stage_rows, f.rows - r0), cut.lane, cut.lanes) : 0;
                    sum_rows<T, E>(rows + (uint32_t)cut.lane * pitch + cc * (E * sizeof(T)), more, (uint32_t)cut.lanes * pitch, n, K, s1, s2);
                    n += more;
                    if (t0 + cut.cols >= CC) at.release(p, fs);
                }
                lane_stats(n, K, s1, s2, lane_mean + threadIdx.x * E, lane_m2 + threadIdx.x * E);
                if ((met = flow_sync_any(at.failed))) break;
                join_lanes<kFlowThreads>(lane_mean, lane_m2, cut.cols * E, cut.lanes, f.rows);
                flow_sync();
                // a group's channels of this tile, joined with those of the tiles before
                const int c0 = t0 * E, c1 = min((t0 + cut.cols) * E, g.C);
                sum_groups<kFlowThreads>(
                    c0, c1, g.cg,
                    [&](int lo, int c) {  // about the first channel's mean
                        const float d = lane_mean[c - c0] - lane_mean[lo - c0];
                        return make_float2(d, fmaf((float)f.rows * d, d, lane_m2[c - c0]));
                    },
                    [&](int k, int lo, int hi, float2 v) {
                        const float w = (float)(hi - lo), off = v.x / w, cnt = (float)f.rows * w;
                        float m = lane_mean[lo - c0] + off, m2 = at_least_0(v.y - (float)f.rows * v.x * off);
                        if (lo > k * g.cg) {
                            const float2 a = acc[k];
                            const float na = (float)f.rows * (float)(lo - k * g.cg), d = m - a.x, share = cnt / (na + cnt);
                            m = a.x + d * share;
                            m2 = a.y + m2 + d * d * (na * share);
                        }
                        if (hi < (k + 1) * g.cg)
                            acc[k] = make_float2(m, m2);
                        else
                            p.part[f.item * g.G + k] = make_float2(m, m2);
                    });
                if (t0 + cut.cols < CC) flow_sync();
            }
            if (met) break;
            flow_tell(fs, at, f.item);
            continue;
        }
        float minus_mean[E], f_[E], beta[E];
        const float2 *stat = reinterpret_cast<const float2 *>(ring + (size_t)at.stage * p.stage_bytes + p.offset[3] + addr_mod16(p.stat + (int64_t)f.b * g.G));
        // (in the piece's first stage: a piece of one tile has its constants from there)
        auto constants = [&](int cc) {
            float gamma[E];
            groups_v(stat, cc * E, g.cg, g.magic, minus_mean, f_);
            params_v<T>(g.gamma, g.w32, cc * E, 1.f, gamma);
            params_v<T>(g.beta, g.w32, cc * E, 0.f, beta);
            mul_v(f_, gamma, f_);
        };
        for (int r0 = 0; r0 < f.rows; r0 += p.stage_rows) {
            if (r0 > 0 && !at.more(fs, ticket)) break;
            const int64_t first = f.first + r0;
            const uint32_t stage = ring0 + (uint32_t)at.stage * p.stage_bytes + addr_mod16(static_cast<const char *>(g.x) + first * pitch);
            const int rows = min(p.stage_rows, f.rows - r0);
            for (int t0 = 0; t0 < CC; t0 += cut.cols) {
                const int cc = t0 + cut.col;
                if (!cut.in || cc >= CC) continue;
                if (r0 == 0 || CC > cut.cols) constants(cc);
                uint32_t from = stage + (uint32_t)cut.lane * pitch + cc * (E * sizeof(T));
                const uint32_t step = (uint32_t)cut.lanes * pitch;
                const int64_t out_step = (int64_t)cut.lanes * g.C;
                int64_t row = first + cut.lane;
                T *out = static_cast<T *>(g.out) + row * g.C + cc * E;
#pragma unroll 2
                for (int n = rows_of_lane(rows, cut.lane, cut.lanes); n > 0; --n, from += step, out += out_step, row += cut.lanes) {
                    float v[E], z[E];
                    const Vals<T, E> raw = held_chunk<T, E>(from);
                    raw.get(v);
                    gn_value<T, ACT>(v, minus_mean, f_, beta, z);
                    Vals<T, E> o;
                    o.set(z);
                    o.store(out);
                    if constexpr (KEEP)
                        keep_chunk<T, E>(raw.u, true, block_lanes<E>(), g.codes + row * g.C + cc * E, g.scales + row * (g.C / kBlock8) + cc * E / kBlock8);
                }
            }
            at.release(p, fs);
        }
    }
    flow_end(p, fs, at, met);
}

template <typename T, int E, int ACT, bool KEPT>
__global__ void __launch_bounds__(kFlowAll, kFlowCtas) gn_bwd_flow(const FlowParams p) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(8) FlowShared fs;
    float *lane_a = reinterpret_cast<float *>(ring + (size_t)p.depth * p.stage_bytes), *lane_s = lane_a + kFlowThreads * E;
    float2 *acc = reinterpret_cast<float2 *>(lane_s + kFlowThreads * E);  // [G]
    const GnParams &g = p.g;
    flow_setup(p, fs);
    constexpr int XE = KEPT ? 1 : (int)sizeof(T);  // bytes of a value of x
    const uint32_t pitch = (uint32_t)g.C * sizeof(T), xpitch = (uint32_t)g.C * XE, spitch = (uint32_t)((g.C + kBlock8 - 1) / kBlock8);
    const char *xsrc = KEPT ? reinterpret_cast<const char *>(g.codes_in) : static_cast<const char *>(g.x);
    if (threadIdx.x >= kFlowThreads) {
        if (threadIdx.x == kFlowThreads) {
            if constexpr (KEPT) {
                const void *const src[3] = {xsrc, g.dy, g.scales_in};
                const uint32_t row[3] = {xpitch, pitch, spitch};
                flow_copies<3>(p, fs, ring, src, row);
            } else {
                const void *const src[2] = {xsrc, g.dy};
                const uint32_t row[2] = {xpitch, pitch};
                flow_copies<2>(p, fs, ring, src, row);
            }
        } else if (threadIdx.x >= kFlowThreads + 32) {
            auto join = [&](const float2 *from, int n, float, int, float) {
                float2 m = make_float2(0.f, 0.f);
                for (int i0 = 0; i0 < n; i0 += kFlowFan) {
                    float2 v[kFlowFan];
#pragma unroll
                    for (int i = 0; i < kFlowFan; ++i) v[i] = __ldcg(from + min(i0 + i, n - 1) * g.G);
#pragma unroll
                    for (int i = 0; i < kFlowFan; ++i)
                        if (i0 + i < n) m = add2(m, v[i]);
                }
                return m;
            };
            flow_join(p, fs, join, [&](int b, int k, float2 m) {
                const float n = (float)g.S * (float)g.cg;
                p.stat[(int64_t)b * g.G + k] = make_float2(-m.x / n, -m.y / n);
            });
        }
        return;
    }
    const int CC = g.C / E;
    const Cut cut(CC, kFlowThreads);
    const uint32_t ring0 = smem_u32(ring);
    // A chunk column's places in a stage, from row to row.
    struct Walk {
        uint32_t x, d, s;
    };
    auto walk = [&](int stage, int64_t first, int cc) {
        const uint32_t at = ring0 + (uint32_t)stage * p.stage_bytes;
        return Walk{at + addr_mod16(xsrc + first * xpitch) + (uint32_t)cut.lane * xpitch + cc * (E * XE),
                    at + p.offset[1] + addr_mod16(static_cast<const char *>(g.dy) + first * pitch) + (uint32_t)cut.lane * pitch + cc * (E * (uint32_t)sizeof(T)),
                    KEPT ? at + p.offset[2] + addr_mod16(g.scales_in + first * spitch) + (uint32_t)cut.lane * spitch + cc * E / kBlock8 : 0u};
    };
    const Walk step{(uint32_t)cut.lanes * xpitch, (uint32_t)cut.lanes * pitch, (uint32_t)cut.lanes * spitch};
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
    FlowStages at{0, 0u, false};
    bool met = false;
    for (int64_t ticket; (ticket = at.wait(fs)) >= 0;) {
        const FlowPiece f(p, ticket);
        auto constants = [&](int cc, float (&minus_mean)[E], float (&rstd)[E], float (&gamma)[E], float (&beta)[E]) {
            const int64_t of = (int64_t)f.b * g.G;
            auto group = [&](int c) { return g.magic ? (int)__umulhi((uint32_t)c, g.magic) : c; };
            if (g.cg % E == 0) {
                const int64_t k = of + group(cc * E);
                fill_v(-g.mean[k], minus_mean);
                fill_v(g.rstd[k], rstd);
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const int64_t k = of + group(cc * E + i);
                    minus_mean[i] = -g.mean[k];
                    rstd[i] = g.rstd[k];
                }
            }
            params_v<T>(g.gamma, g.w32, cc * E, 1.f, gamma);
            params_v<T>(g.beta, g.w32, cc * E, 0.f, beta);
        };
        if (!f.normalise) {
            float *out = g.parts ? g.parts + f.item * 2 * g.C : nullptr;
            for (int t0 = 0; t0 < CC; t0 += cut.cols) {
                const int cc = t0 + cut.col;
                const bool in = cut.in && cc < CC;
                float a[E], s[E], minus_mean[E], rstd[E], gamma[E], beta[E];
                fill_v(0.f, a);
                fill_v(0.f, s);
                if (in) constants(cc, minus_mean, rstd, gamma, beta);
                for (int r0 = 0; r0 < f.rows; r0 += p.stage_rows) {
                    if (r0 > 0 && !at.more(fs, ticket)) break;
                    Walk w = walk(at.stage, f.first + r0, cc);
                    const int n = in ? rows_of_lane(min(p.stage_rows, f.rows - r0), cut.lane, cut.lanes) : 0;
#pragma unroll 2
                    for (int k = 0; k < n; ++k) {
                        float xhat[E], u[E];
                        chunk(w, minus_mean, rstd, gamma, beta, xhat, u);
                        fma_v(u, xhat, a, a);
                        add_v(s, u, s);
                    }
                    if (t0 + cut.cols >= CC) at.release(p, fs);
                }
                put_v(lane_a + threadIdx.x * E, a);
                put_v(lane_s + threadIdx.x * E, s);
                if ((met = flow_sync_any(at.failed))) break;
                const int width = cut.cols * E, c0 = t0 * E, c1 = min(c0 + width, g.C);
                for (int c = threadIdx.x; c < c1 - c0; c += kFlowThreads) {
                    float ta = lane_a[c], ts = lane_s[c];
#pragma unroll 8
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
                flow_sync();
                sum_groups<kFlowThreads>(
                    c0, c1, g.cg, [&](int, int c) { return make_float2(lane_s[c - c0], lane_a[c - c0]); },
                    [&](int k, int lo, int hi, float2 m) {
                        if (lo > k * g.cg) m = add2(acc[k], m);
                        if (hi < (k + 1) * g.cg)
                            acc[k] = m;
                        else
                            p.part[f.item * g.G + k] = m;
                    });
                if (t0 + cut.cols < CC) flow_sync();
            }
            if (met) break;
            flow_tell(fs, at, f.item);
            continue;
        }
        const float2 *stat = reinterpret_cast<const float2 *>(ring + (size_t)at.stage * p.stage_bytes + p.offset[3] + addr_mod16(p.stat + (int64_t)f.b * g.G));
        float minus_mean[E], rstd[E], gamma[E], beta[E], m1[E], m2[E];
        for (int r0 = 0; r0 < f.rows; r0 += p.stage_rows) {
            if (r0 > 0 && !at.more(fs, ticket)) break;
            const int64_t first = f.first + r0;
            const int rows = min(p.stage_rows, f.rows - r0);
            for (int t0 = 0; t0 < CC; t0 += cut.cols) {
                const int cc = t0 + cut.col;
                if (!cut.in || cc >= CC) continue;
                if (r0 == 0 || CC > cut.cols) {
                    constants(cc, minus_mean, rstd, gamma, beta);
                    groups_v(stat, cc * E, g.cg, g.magic, m1, m2);
                }
                Walk w = walk(at.stage, first, cc);
                const int64_t out_step = (int64_t)cut.lanes * g.C;
                T *to = static_cast<T *>(g.out) + (first + cut.lane) * g.C + cc * E;
#pragma unroll(E == 8 ? 1 : 2)
                for (int n = rows_of_lane(rows, cut.lane, cut.lanes); n > 0; --n, to += out_step) {
                    float xhat[E], u[E];
                    chunk(w, minus_mean, rstd, gamma, beta, xhat, u);
                    gn_dx(xhat, u, rstd, gamma, m1, m2);
                    Vals<T, E> o;
                    o.set(u);
                    o.store(to);
                }
            }
            at.release(p, fs);
        }
    }
    flow_end(p, fs, at, met);
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

// (keeping x in the same pass: chunks only)
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
// A kernel by chunks of `chunk` values.
template <typename T> static const void *gn_flow_t(bool backward, int chunk, int act, bool kept) {
    if constexpr (sizeof(T) == 2) {
        if (chunk == 8) return gn_flow_e<T, 8>(backward, act, kept);
    }
    return chunk == 4 ? gn_flow_e<T, 4>(backward, act, kept) : gn_flow_e<T, 1>(backward, act, kept);
}

}  // namespace rmsn
