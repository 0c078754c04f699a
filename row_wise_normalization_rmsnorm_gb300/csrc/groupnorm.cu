// groupnorm.cu -- entry points of group norm (declared in include/rmsnorm.h):
// argument checks, the cut of the work, the workspace and the launches.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>

#include "groupnorm_flow.cuh"
#include "groupnorm_held.cuh"
#include "head_rows.h"
#include "plans.h"
#include "train_rows.h"

namespace rmsn {

static const void *gn_flow(int base, bool backward, int chunk, int act, bool kept) {
    return base == RMSNORM_BF16 ? gn_flow_bf16(backward, chunk, act, kept)
           : base == RMSNORM_F16 ? gn_flow_f16(backward, chunk, act, kept)
                                 : gn_flow_f32(backward, chunk, act, kept);
}

struct GnCall {
    int64_t B, S, C;
    int G, act, dt;
    bool backward;
    bool kept;  // backward: x comes as codes; forward: codes are written in the same pass
    int chunk;  // values of a chunk: 8 or 4 of them, or single ones
};

// The largest power of two, up to 16, that all addresses are multiples of.
static int align_of(std::initializer_list<const void *> rows) {
    uintptr_t all = 16;
    for (const void *p : rows) all |= (uintptr_t)p;
    return (int)(all & (~all + 1));
}

// The widest chunk, up to 16 bytes, that the rows (and the codes that are read)
// are whole numbers of, on its boundary.
static int chunk_of(int64_t C, int es, int row_align, int code_align) {
    for (int chunk = 16 / es; chunk >= 4; chunk /= 2)
        if (C % chunk == 0 && row_align >= chunk * es && code_align >= chunk) return chunk;
    return 1;
}

// A call whose arrays lie on these boundaries. The forward keeps x in its own
// pass where rows are whole blocks of chunks, else by a launch of ckpt8_pack.
static GnCall gn_call(int64_t B, int64_t S, int64_t C, int64_t G, int act, int dt, bool backward, bool kept, int row_align, int code_align) {
    GnCall c{B, S, C, (int)G, act, dt, backward, kept, chunk_of(C, bytes_of(dt), row_align, backward && kept ? code_align : 16)};
    if (!backward) c.kept = kept && c.chunk > 1 && C % kBlock8 == 0 && code_align >= c.chunk;
    return c;
}

static const void *gn_held(int base, bool backward, int chunk, int act, bool kept) {
    return base == RMSNORM_BF16 ? gn_held_bf16(backward, chunk, act, kept)
           : base == RMSNORM_F16 ? gn_held_f16(backward, chunk, act, kept)
                                 : gn_held_f32(backward, chunk, act, kept);
}

// The cut of the one-launch kernels: a cluster of `ctas` CTAs a unit of K
// groups of a sample. `ctas` is 0 where no cut fits.
struct GnHeld {
    int ctas, K, W, rows;
    uint32_t slab[2], scales;
    size_t smem;
};

constexpr size_t kHeldSmem = 112 * 1024;  // of a CTA: two an SM
constexpr int kHeldGroups = 256;          // of a cluster at most

// A device as the plans see it: its SMs, and the CTAs of the largest cluster
// (1, 2, 4, 8 or 16) that it holds with a held CTA's threads and shared memory.
struct GnDevice {
    int sms, cluster;
};

// (never launched: what the runtime is asked about)
__global__ void __launch_bounds__(kHeldThreads, 2) gn_cluster_room() {}

// The current device, asked once; a cudaError_t.
static int gn_device(GnDevice &on, int **status) {
    static std::mutex mu;
    static int most[64];
    int dev = 0;
    const int e = current_device(&on.sms, status, &dev);
    if (e != 0) return e;
    std::lock_guard<std::mutex> lk(mu);
    if (most[dev] == 0) {
        auto *kernel = gn_cluster_room;
        most[dev] = 1;
        const bool ok = allow_staged_smem(reinterpret_cast<const void *>(kernel)) == 0;
        const bool wide = ok && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
        for (int size = wide ? kHeldCtas : 8; ok && size > 1 && most[dev] == 1; size /= 2) {
            LaunchCfg lc((unsigned)(size * on.sms), kHeldThreads, kHeldSmem, nullptr, (unsigned)size, false);
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, kernel, &lc.cfg) == cudaSuccess && n > 0) most[dev] = size;
        }
        (void)cudaGetLastError();
    }
    on.cluster = most[dev];
    return 0;
}

// What a cut needs; false: it does not fit.
static bool held_cut(const GnCall &c, int K, int ctas, GnHeld &h) {
    const int es = bytes_of(c.dt), E = c.chunk, cg = (int)(c.C / c.G);
    const int64_t W = (int64_t)K * cg, rows = (c.S + ctas - 1) / ctas;
    const bool span = K < c.G;
    // a span is whole chunks, of 64 bytes a row at least; kept in whole blocks of 32
    if (W > 4096 || c.B * (c.G / K) * ctas > 0x7fffffffLL || (span && (c.chunk == 1 || W % E != 0 || W * es < 64))) return false;
    if (!c.backward && c.kept && W % kBlock8 != 0) return false;
    const bool codes = c.backward && c.kept;
    const int xb = codes ? 1 : es;
    auto up = [](int64_t n) { return (n + 15) / 16 * 16; };
    const int64_t x = up(rows * W * xb + 16), d = c.backward ? up(rows * W * es + 16) : 0;
    const int64_t sc = codes ? up(rows * (W / kBlock8 + 2)) : 0;
    const int64_t fixed = kHeldThreads * E * 8 + W * 8 + (int64_t)ctas * K * 8 + K * 16;  // (statistics: the CTAs', the cluster's, this CTA's)
    if (x + d + sc + fixed > (int64_t)kHeldSmem) return false;
    h = GnHeld{ctas, K, (int)W, (int)rows, {(uint32_t)x, (uint32_t)d}, (uint32_t)sc, (size_t)(x + d + sc + fixed)};
    return true;
}

// The cheapest cut by estimate: rounds of the CTAs that an SM holds at once
// (two), at 4.5 us each, and the bytes at the rate of memory, those of a span
// that begins or ends inside a 32-byte sector counted with the whole sector.
// (The gradient of 8 x 4096 x 320: spans of 80 bytes in clusters of 8 take 33
// us, of 160 bytes in clusters of 16 39, the flow 57.)
static GnHeld held_plan(const GnCall &c, const GnDevice &on) {
    const int sms = on.sms;
    GnHeld best{0, 0, 0, 0, {0, 0}, 0, 0};
    double least = 0;
    const int es = bytes_of(c.dt);
    for (int K = 1; K <= c.G && K <= kHeldGroups; ++K) {
        if (c.G % K != 0) continue;
        for (int n = 1; n <= on.cluster; n *= 2) {
            GnHeld h;
            if ((n > 1 && (c.S + n - 1) / n * (n - 1) >= c.S) || !held_cut(c, K, n, h)) continue;
            const double row = (double)h.W * es, sectors = K == c.G || (h.W * es) % 32 == 0 ? row : row + 32;
            const double bytes = (double)c.B * c.S * c.C * es * (c.backward ? 3 : 2) * (sectors / row);
            // clusters of 16 leave SMs without a CTA where a GPU's groups of SMs are no multiple of 8
            const double ctas = (double)c.B * (c.G / K) * n, places = 2.0 * sms * (n == 16 ? 0.73 : n == 8 ? 0.94 : 1.0);
            const double rounds = std::ceil(ctas / places);
            const double share = ctas < sms ? sms / ctas : 1.0;  // SMs without a CTA
            const double cost = 4.5 * rounds + (n > 1 ? 0.5 : 0.0) + bytes * share / 6.7e6;
            if (best.ctas == 0 || cost < least) {
                best = h;
                least = cost;
            }
        }
    }
    return best;
}

// Workspace of the one-launch gradient: a CTA's channel sums.
static size_t held_bytes(const GnCall &c, const GnHeld &h) { return ((size_t)c.B * h.ctas * 2 * c.C * 4 + 255) / 256 * 256; }

// The cut of the flow: pieces of `rows` places of a sample, stages of
// `stage_rows`.
struct GnFlow {
    int rows, pieces, fans, lag, grid, folds, stage_rows, depth;
    uint32_t offset[4], stage_bytes;
    size_t smem;
    size_t state, part, fan, stat, parts, folded, bytes;  // workspace offsets (state_bytes of zeros first)
    size_t state_bytes;
};

// Values of a chunk of the gradient's flow: with 8 a thread's constants of 8
// channels spill, with 4 a row of more than 1024 channels is several tiles.
static int flow_chunk(int chunk, int64_t C) { return chunk > 4 && C <= 4 * kFlowThreads ? 4 : chunk; }

// Bytes of a stage, and of a piece at most: small pieces are summed, joined and
// normalised sooner, large ones cost fewer joins. (256 x 256 x 256, 8 images:
// pieces of 128 KB and a lag of one and a half rounds of the CTAs 144 us, of 256
// KB and one round 154, of 64 KB and one round 158. The gradient, which reads two
// tensors a piece: 281 and 267 with the first two.)
constexpr int64_t kFlowStage = 28 << 10, kFlowPiece = 128 << 10, kFlowBwdPiece = 256 << 10;
constexpr size_t kFlowSmem = 226 * 1024 / kFlowCtas, kFlowSmemMost = 224 * 1024;  // of a CTA; of the only one on an SM

static GnFlow flow_plan(const GnCall &c, int sms) {
    GnFlow f;
    const bool codes = c.backward && c.kept;
    const int es = bytes_of(c.dt), E = c.chunk, xb = codes ? 1 : es;
    const int64_t CC = c.C / E, tiles = (CC + kFlowThreads - 1) / kFlowThreads,
                  cols = tiles > 1 ? ((CC + tiles - 1) / tiles + 7) / 8 * 8 : CC, lanes = kFlowThreads / cols;
    const int64_t nb = codes ? (c.C + kBlock8 - 1) / kBlock8 : 0;
    f.smem = 2 * sizeof(float) * kFlowThreads * E + (size_t)c.G * sizeof(float2);
    // stages: three at least, of whole turns of the lanes, where a row is small enough
    const int64_t row = c.C * (c.backward ? xb + es : es) + nb;
    int64_t room = (int64_t)kFlowSmem - 1024 - (int64_t)f.smem;
    auto bytes = [&](int64_t rows) {  // of a stage: the 16-byte blocks that hold its rows
        auto up = [](int64_t n) { return (n + 30) / 16 * 16; };
        f.offset[0] = 0;
        f.offset[1] = (uint32_t)up(rows * c.C * xb);
        f.offset[2] = f.offset[1] + (uint32_t)(c.backward ? up(rows * c.C * es) : 0);
        f.offset[3] = f.offset[2] + (uint32_t)(codes ? up(rows * nb) : 0);
        f.stage_bytes = f.offset[3] + (uint32_t)up((int64_t)c.G * 8);
        return (int64_t)f.stage_bytes;
    };
    int64_t rows = std::max<int64_t>(1, kFlowStage / row / lanes) * lanes;
    while (rows > 1 && 3 * bytes(rows) > room) rows = rows > lanes ? std::max<int64_t>(rows / 2 / lanes, 1) * lanes : rows / 2;
    // (rows of ROWS_MAX_CHANNELS in one CTA an SM: two stages fit, but for the fp32 gradient with
    // more than 3900 groups, whose statistics are as large as a row: one, 98 KB)
    if (2 * bytes(rows) > room) room = (int64_t)kFlowSmemMost - (int64_t)f.smem;
    f.stage_rows = (int)rows;
    f.depth = (int)std::min<int64_t>(kFlowStagesMost, room / std::max<int64_t>(1, bytes(rows)));
    f.grid = kFlowCtas * sms;
    // pieces: the sums' joining is a cost a piece, so several stages where a row is one tile
    // (and whole turns of the lanes fit a stage), but two pieces for every CTA where there are rows enough
    int64_t turns = 1;
    if (tiles == 1 && rows % lanes == 0)
        while (turns < 64 && 2 * turns * rows * row <= (c.backward ? kFlowBwdPiece : kFlowPiece) && c.S * c.B >= 4 * turns * rows * f.grid) turns *= 2;
    rows *= turns;
    while ((c.S + rows - 1) / rows > 65535 && tiles == 1 && rows % lanes == 0) rows *= 2;
    f.rows = (int)std::min<int64_t>(rows, c.S);
    f.pieces = (int)((c.S + f.rows - 1) / f.rows);
    f.lag = c.backward ? f.grid : f.grid * 3 / 2;
    f.grid = (int)std::min<int64_t>(f.grid, c.B * f.pieces);
    if (c.B * f.pieces <= f.grid) f.lag = 0;  // one turn of the CTAs: nothing to put between
    f.smem += (size_t)f.depth * f.stage_bytes;
    size_t at = 0;
    auto take = [&at](size_t n) {
        const size_t a = at;
        at += (n + 255) / 256 * 256;
        return a;
    };
    f.fans = (f.pieces + kFlowFan - 1) / kFlowFan;
    f.state_bytes = (size_t)(2 + (2 + f.fans) * c.B) * 4;
    f.state = take(f.state_bytes);
    f.part = take((size_t)c.B * f.pieces * c.G * sizeof(float2));
    f.fan = take((size_t)c.B * f.fans * c.G * sizeof(float2));
    f.stat = take((size_t)c.B * c.G * sizeof(float2));
    f.parts = f.folded = at;
    f.folds = 0;
    if (c.backward) {
        f.parts = take((size_t)c.B * f.pieces * 2 * c.C * 4);
        if (c.B * f.pieces > 512) f.folds = 64;  // (the finalizer sums 32 groups of rows, one after the other)
        f.folded = take((size_t)f.folds * 2 * c.C * 4);
    }
    f.bytes = at;
    return f;
}

// The cut of a call and the workspace that it takes: what the calls launch by
// and what the queries answer from.
struct GnCut {
    GnCall c;  // with the chunk of the kernels that run
    GnHeld h;
    GnFlow f;  // where h.ctas is 0
    size_t bytes;
};
static GnCut gn_cut(const GnCall &c, const GnDevice &on) {
    GnCut k;
    std::memset(&k, 0, sizeof k);
    k.c = c;
    k.h = held_plan(c, on);
    if (k.h.ctas) {
        k.bytes = c.backward ? held_bytes(c, k.h) : 0;
    } else {
        if (c.backward) k.c.chunk = flow_chunk(c.chunk, c.C);
        k.f = flow_plan(k.c, on.sms);
        k.bytes = k.f.bytes;
    }
    return k;
}

static bool gn_sizes(int64_t B, int64_t S, int64_t C, int64_t G, int act, int dt) {
    const int base = dt & ~RMSNORM_WEIGHT_F32;
    if (base != RMSNORM_F32 && base != RMSNORM_BF16 && base != RMSNORM_F16) return false;
    if (B < 0 || S < 0 || C < 1 || C > ROWS_MAX_CHANNELS || G < 1 || C % G != 0) return false;
    if (B > 0x7fffffffLL || S > 0x7fffffffLL) return false;
    if (B > 0 && S > INT64_MAX / 8 / C / B) return false;
    return act >= kActNone && act <= kActGelu;
}

// dgamma and dbeta from rows of both ([n, 2 C]).
static int gn_finalize(int base, int w32, const float *rows, int n, int64_t C, void *dgamma, void *dbeta, int sms, cudaStream_t s) {
    auto *fin = base == RMSNORM_F32 || w32 ? launch_dw_finalize_f32 : base == RMSNORM_BF16 ? launch_dw_finalize_bf16 : launch_dw_finalize_f16;
    return fin(rows, n, (int)(2 * C), dgamma, dbeta, (int)C, 0, s, false, sms);
}

static rmsnorm_status_t gn_run_held(const GnParams &g, const GnCall &c, const GnHeld &h, void *dgamma, void *dbeta, int sms,
                                    int *status, cudaStream_t s) {
    const int base = base_of(c.dt);
    HeldParams p;
    std::memset(&p, 0, sizeof p);
    p.g = g;
    p.g.rows = h.rows;
    if (c.backward && !dgamma && !dbeta) p.g.parts = nullptr;
    p.ctas = h.ctas, p.W = h.W, p.K = h.K, p.spans = c.G / h.K;
    p.slab[0] = h.slab[0], p.slab[1] = h.slab[1], p.scales = h.scales;
    p.status = status;
    const void *k = gn_held(base, c.backward, c.chunk, c.act, c.backward ? c.kept : g.codes != nullptr);
    if (h.ctas > 8) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return head_cuda_fail((int)e);
    }
    void *args[] = {&p};
    const int64_t grid = c.B * p.spans * h.ctas;
    int e = launch(k, (unsigned)grid, 1, kHeldThreads, h.smem, args, s, (unsigned)h.ctas);
    if (e == 0 && c.backward && (dgamma || dbeta)) e = gn_finalize(base, g.w32, g.parts, (int)(c.B * h.ctas), c.C, dgamma, dbeta, sms, s);
    return e == 0 ? RMSNORM_SUCCESS : head_cuda_fail(e);
}

// A sample whose pieces are never joined, and the polls that are made for it.
struct GnLose {
    int64_t sample;
    uint32_t polls;
};

static rmsnorm_status_t gn_run_flow(const GnParams &g, const GnCall &c, const GnFlow &f, char *w, void *dgamma, void *dbeta,
                                    int sms, int *status, cudaStream_t s, const GnLose *lose = nullptr) {
    const int base = base_of(c.dt);
    if (f.depth < 1) return RMSNORM_ERR_UNSUPPORTED;  // (no size that is taken: rows of ROWS_MAX_CHANNELS have a stage)
    FlowParams p;
    std::memset(&p, 0, sizeof p);
    p.g = g;
    p.g.rows = f.rows;
    const bool sums = c.backward && (dgamma || dbeta);
    p.g.parts = sums ? reinterpret_cast<float *>(w + f.parts) : nullptr;
    p.pieces = f.pieces, p.lag = f.lag;
    p.tickets = 2 * (c.B * f.pieces + f.pieces + f.lag);
    p.stage_rows = f.stage_rows, p.depth = f.depth, p.stage_bytes = f.stage_bytes;
    for (int i = 0; i < 4; ++i) p.offset[i] = f.offset[i];
    p.state = reinterpret_cast<uint32_t *>(w + f.state);
    p.fans = f.fans;
    p.part = reinterpret_cast<float2 *>(w + f.part), p.fan = reinterpret_cast<float2 *>(w + f.fan), p.stat = reinterpret_cast<float2 *>(w + f.stat);
    p.stat_limit = lose ? lose->polls : kFlowStatLimit;
    p.status = status;
    int e = (int)cudaMemsetAsync(p.state, 0, f.state_bytes, s);
    if (e == 0 && lose) e = (int)cudaMemsetAsync(p.state + 2 + c.B + lose->sample, 0x40, 4, s);  // a count that the sample's pieces do not end
    void *args[] = {&p};
    if (e == 0)
        e = launch(gn_flow(base, c.backward, c.chunk, c.act, c.backward ? c.kept : g.codes != nullptr), (unsigned)f.grid, 1, kFlowAll,
                   f.smem, args, s, 1);
    if (e == 0 && sums) {
        const float *in = p.g.parts;
        int64_t n = c.B * f.pieces;
        if (f.folds) {
            float *out = reinterpret_cast<float *>(w + f.folded);
            int width = (int)(2 * c.C);
            void *fargs[] = {&in, &out, &n, &width};
            e = launch((const void *)gn_fold, (unsigned)((width + 255) / 256), (unsigned)f.folds, 256, 0, fargs, s);
            in = out;
            n = f.folds;
        }
        if (e == 0) e = gn_finalize(base, g.w32, in, (int)n, c.C, dgamma, dbeta, sms, s);
    }
    return e == 0 ? RMSNORM_SUCCESS : head_cuda_fail(e);
}

// The most that any alignment takes, with x kept in 8 bits or not.
static size_t gn_workspace(int64_t B, int64_t S, int64_t C, int64_t G, int dt, bool backward, const GnDevice &on) {
    size_t most = 0;
    for (int row = 16; row > 0; row /= 2)
        for (int code = 16; code > 0; code /= 2)
            for (int kept = 0; kept < 2; ++kept) {
                // each cut once: of the least alignment that gives its chunk
                const GnCall c = gn_call(B, S, C, G, 0, dt, backward, kept != 0, row, code);
                if (row > 1 && c.chunk == gn_call(B, S, C, G, 0, dt, backward, kept != 0, row / 2, code).chunk) continue;
                if (code > 1) {
                    const GnCall less = gn_call(B, S, C, G, 0, dt, backward, kept != 0, row, code / 2);
                    if (c.chunk == less.chunk && c.kept == less.kept) continue;
                }
                most = std::max(most, gn_cut(c, on).bytes);
            }
    return most;
}

}  // namespace rmsn

using namespace rmsn;

extern "C" rmsnorm_status_t groupnorm_fwd(const void *x, const void *gamma, const void *beta, void *y, float *mean,
                                          float *rstd, void *codes, uint8_t *scales, void *workspace,
                                          size_t workspace_bytes, int64_t B, int64_t S, int64_t C, int64_t G,
                                          rmsnorm_act_t act, rmsnorm_dtype_t dt, float eps, rmsnorm_stream_t stream) {
    if (!gn_sizes(B, S, C, G, act, dt) || !std::isfinite(eps) || eps < 0.f || (codes == nullptr) != (scales == nullptr))
        return RMSNORM_ERR_INVALID_ARG;
    if (B == 0) return RMSNORM_SUCCESS;
    if (G > ROWS_MAX_GROUPS) return RMSNORM_ERR_UNSUPPORTED;
    const int base = dt & ~RMSNORM_WEIGHT_F32, es = base == RMSNORM_F32 ? 4 : 2;
    const uintptr_t ws = base == RMSNORM_F32 || (dt & RMSNORM_WEIGHT_F32) ? 4 : 2;
    if (!mean || !rstd || !on(mean, 4) || !on(rstd, 4) || !on(gamma, ws) || !on(beta, ws)) return RMSNORM_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (S == 0) return zeros({{mean, (size_t)(B * G) * 4}, {rstd, (size_t)(B * G) * 4}}, s);
    if (!x || !y || !on(x, es) || !on(y, es)) return RMSNORM_ERR_INVALID_ARG;
    GnDevice here;
    int *status = nullptr;
    const int e = gn_device(here, &status);
    if (e != 0) return head_cuda_fail(e);
    const int sms = here.sms;
    const GnCut k = gn_cut(gn_call(B, S, C, G, act, dt, false, codes != nullptr, align_of({x, y}), align_of({codes})), here);
    GnParams p;
    std::memset(&p, 0, sizeof p);
    p.x = x, p.gamma = gamma, p.beta = beta, p.out = y, p.mean = mean, p.rstd = rstd;
    p.S = S, p.B = (int)B, p.C = (int)C, p.G = (int)G, p.cg = (int)(C / G);
    p.magic = p.cg == 1 ? 0u : (uint32_t)(((1ull << 32) + p.cg - 1) / p.cg);
    p.w32 = (dt & RMSNORM_WEIGHT_F32) || base == RMSNORM_F32, p.eps = eps;
    if (k.c.kept) p.codes = static_cast<uint8_t *>(codes), p.scales = scales;
    if (codes && !k.c.kept) {  // first: y may be x
        const rmsnorm_status_t st = ckpt8_pack(x, codes, scales, B * S, C, (rmsnorm_dtype_t)base, stream);
        if (st != RMSNORM_SUCCESS) return st;
    }
    if (k.h.ctas) return gn_run_held(p, k.c, k.h, nullptr, nullptr, sms, status, s);
    return with_workspace(workspace, workspace_bytes, k.bytes, s,
                          [&](char *w) { return gn_run_flow(p, k.c, k.f, w, nullptr, nullptr, sms, status, s); });
}

extern "C" rmsnorm_status_t groupnorm_bwd(const void *dy, const void *x, const void *codes, const uint8_t *scales,
                                          const void *gamma, const void *beta, const float *mean, const float *rstd,
                                          void *dx, void *dgamma, void *dbeta, void *workspace, size_t workspace_bytes,
                                          int64_t B, int64_t S, int64_t C, int64_t G, rmsnorm_act_t act,
                                          rmsnorm_dtype_t dt, rmsnorm_stream_t stream) {
    if (!gn_sizes(B, S, C, G, act, dt) || (codes == nullptr) != (scales == nullptr) || (dgamma && !gamma))
        return RMSNORM_ERR_INVALID_ARG;
    const int base = dt & ~RMSNORM_WEIGHT_F32, es = base == RMSNORM_F32 ? 4 : 2;
    const uintptr_t ws = base == RMSNORM_F32 || (dt & RMSNORM_WEIGHT_F32) ? 4 : 2;
    if (!on(gamma, ws) || !on(beta, ws) || !on(dgamma, ws) || !on(dbeta, ws)) return RMSNORM_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (B == 0 || S == 0) return zeros({{dgamma, (size_t)C * ws}, {dbeta, (size_t)C * ws}}, s);
    if (G > ROWS_MAX_GROUPS) return RMSNORM_ERR_UNSUPPORTED;
    if (!dy || !dx || !mean || !rstd || (x == nullptr) == (codes == nullptr)) return RMSNORM_ERR_INVALID_ARG;
    if (!on(dy, es) || !on(dx, es) || !on(x, es) || !on(mean, 4) || !on(rstd, 4)) return RMSNORM_ERR_INVALID_ARG;
    GnDevice here;
    int *status = nullptr;
    const int e = gn_device(here, &status);
    if (e != 0) return head_cuda_fail(e);
    const int sms = here.sms;
    const GnCut k = gn_cut(gn_call(B, S, C, G, act, dt, true, codes != nullptr, align_of({dy, dx, x}), align_of({codes})), here);
    GnParams p;
    std::memset(&p, 0, sizeof p);
    p.x = x, p.dy = dy, p.codes_in = static_cast<const uint8_t *>(codes), p.scales_in = scales;
    p.gamma = gamma, p.beta = beta, p.out = dx, p.mean = const_cast<float *>(mean), p.rstd = const_cast<float *>(rstd);
    p.S = S, p.B = (int)B, p.C = (int)C, p.G = (int)G, p.cg = (int)(C / G);
    p.magic = p.cg == 1 ? 0u : (uint32_t)(((1ull << 32) + p.cg - 1) / p.cg);
    p.w32 = (dt & RMSNORM_WEIGHT_F32) || base == RMSNORM_F32;
    return with_workspace(workspace, workspace_bytes, k.bytes, s, [&](char *w) {
        if (!k.h.ctas) return gn_run_flow(p, k.c, k.f, w, dgamma, dbeta, sms, status, s);
        p.parts = reinterpret_cast<float *>(w);
        return gn_run_held(p, k.c, k.h, dgamma, dbeta, sms, status, s);
    });
}

extern "C" rmsnorm_status_t groupnorm_plan_query(int64_t B, int64_t S, int64_t C, int64_t G, rmsnorm_dtype_t dt, int backward,
                                                 int kept, int32_t row_align, int32_t code_align, int32_t num_sms,
                                                 int32_t max_cluster, groupnorm_plan_t *plan) {
    if (!plan || !gn_sizes(B, S, C, G, 0, dt) || num_sms < 0 || row_align < 0 || code_align < 0 || (num_sms > 0 && max_cluster < 1))
        return RMSNORM_ERR_INVALID_ARG;
    if (G > ROWS_MAX_GROUPS) return RMSNORM_ERR_UNSUPPORTED;
    std::memset(plan, 0, sizeof *plan);
    if (B == 0 || S == 0) return RMSNORM_SUCCESS;
    GnDevice on{num_sms, max_cluster < kHeldCtas ? max_cluster : kHeldCtas};
    if (num_sms == 0) {
        const int e = gn_device(on, nullptr);
        if (e != 0) return head_cuda_fail(e);
    }
    if (row_align == 0) {
        plan->workspace_bytes = (int64_t)gn_workspace(B, S, C, G, dt, backward != 0, on);
        return RMSNORM_SUCCESS;
    }
    const GnCut k = gn_cut(gn_call(B, S, C, G, 0, dt, backward != 0, kept != 0, row_align, code_align), on);
    plan->chunk = k.c.chunk, plan->cluster = k.h.ctas, plan->groups = k.h.K;
    plan->rows = k.h.ctas ? k.h.rows : k.f.rows;
    plan->stages = k.h.ctas ? 0 : k.f.depth;
    plan->smem_bytes = (int32_t)(k.h.ctas ? k.h.smem : k.f.smem);
    plan->workspace_bytes = (int64_t)k.bytes;
    return RMSNORM_SUCCESS;
}

extern "C" size_t groupnorm_workspace_bytes(int64_t B, int64_t S, int64_t C, int64_t G, rmsnorm_dtype_t dt, int backward) {
    groupnorm_plan_t plan;
    return groupnorm_plan_query(B, S, C, G, dt, backward, 0, 0, 0, 0, 0, &plan) == RMSNORM_SUCCESS ? (size_t)plan.workspace_bytes : 0;
}

extern "C" rmsnorm_status_t groupnorm_give_up_check(const void *dy, const void *x, float *mean, float *rstd, void *out, int64_t B,
                                                    int64_t S, int64_t C, int64_t G, rmsnorm_dtype_t dt, int64_t sample,
                                                    uint32_t polls, rmsnorm_stream_t stream) {
    if (!gn_sizes(B, S, C, G, 0, dt) || base_of(dt) != dt || B == 0 || S == 0 || G > ROWS_MAX_GROUPS || sample < 0 || sample >= B || polls == 0)
        return RMSNORM_ERR_INVALID_ARG;
    const int es = bytes_of(dt);
    if (!x || !out || !mean || !rstd || !on(x, es) || !on(out, es) || !on(dy, es) || !on(mean, 4) || !on(rstd, 4)) return RMSNORM_ERR_INVALID_ARG;
    GnDevice here;
    int *status = nullptr;
    const int e = gn_device(here, &status);
    if (e != 0) return head_cuda_fail(e);
    const int sms = here.sms;
    GnCall c = gn_call(B, S, C, G, 0, dt, dy != nullptr, false, align_of({dy, x, out}), 16);
    if (dy) c.chunk = flow_chunk(c.chunk, C);
    const GnFlow f = flow_plan(c, sms);
    GnParams p;
    std::memset(&p, 0, sizeof p);
    p.x = x, p.dy = dy, p.out = out, p.mean = mean, p.rstd = rstd;
    p.S = S, p.B = (int)B, p.C = (int)C, p.G = (int)G, p.cg = (int)(C / G);
    p.magic = p.cg == 1 ? 0u : (uint32_t)(((1ull << 32) + p.cg - 1) / p.cg);
    p.eps = 1e-5f;
    const GnLose lose{sample, polls};
    return with_workspace(nullptr, 0, f.bytes, (cudaStream_t)stream, [&](char *w) {
        return gn_run_flow(p, c, f, w, nullptr, nullptr, sms, status, (cudaStream_t)stream, &lose);
    });
}
