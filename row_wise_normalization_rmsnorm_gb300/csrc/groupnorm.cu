// groupnorm.cu -- entry points of group norm (declared in include/rmsnorm.h):
// argument checks, the cut of the work, the workspace and the launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "groupnorm_held.cuh"
#include "head_rows.h"
#include "plans.h"
#include "train_rows.h"

namespace rmsn {

static const void *gn_kernel(int which, int base, bool wide, int act, bool kept) {
    return base == RMSNORM_BF16 ? gn_kernel_bf16(which, wide, act, kept)
           : base == RMSNORM_F16 ? gn_kernel_f16(which, wide, act, kept)
                                 : gn_kernel_f32(which, wide, act, kept);
}

struct GnCall {
    int64_t B, S, C;
    int G, act, dt;
    bool backward, kept, wide;
};

// How a call is cut. A CTA has at most `threads` threads, as rows x channel
// chunks; a sample is `chunks` runs of `rows` rows.
struct GnPlan {
    int threads, rows, chunks, batch;  // batch: samples a launch
    size_t parts, sums, means, bytes;  // workspace offsets
};

static const void *gn_held(int base, bool backward, bool wide, int act, bool kept) {
    return base == RMSNORM_BF16 ? gn_held_bf16(backward, wide, act, kept)
           : base == RMSNORM_F16 ? gn_held_f16(backward, wide, act, kept)
                                 : gn_held_f32(backward, wide, act, kept);
}

// The cut of the one-launch kernels: a cluster of `ctas` CTAs a unit of K
// groups of a sample. `ctas` is 0 where no cut fits.
struct GnHeld {
    int ctas, K, W, rows;
    uint32_t slab[2], scales;
    size_t smem;
};

constexpr size_t kHeldSmem = 112 * 1024;  // of a CTA: two an SM

// What a cut needs; false: it does not fit.
static bool held_cut(const GnCall &c, int K, int ctas, bool keep, GnHeld &h) {
    const int es = bytes_of(c.dt), E = c.wide ? 16 / es : 1, cg = (int)(c.C / c.G);
    const int64_t W = (int64_t)K * cg, rows = (c.S + ctas - 1) / ctas;
    const bool span = K < c.G;
    // a span is whole chunks, of 64 bytes a row at least; kept in whole blocks of 32
    if (W > 4096 || K > 256 || (span && (!c.wide || W % E != 0 || W * es < 64))) return false;
    if (keep && W % kBlock8 != 0) return false;
    const int xb = c.kept ? 1 : es;
    auto up = [](int64_t n) { return (n + 15) / 16 * 16; };
    const int64_t x = up(rows * W * xb + 16), d = c.backward ? up(rows * W * es + 16) : 0;
    const int64_t sc = c.kept ? up(rows * (W / kBlock8 + 2)) : 0;
    const int64_t fixed = kHeldThreads * E * 8 + W * 8 + (int64_t)ctas * K * 8 + K * 16;
    if (x + d + sc + fixed > (int64_t)kHeldSmem) return false;
    h = GnHeld{ctas, K, (int)W, (int)rows, {(uint32_t)x, (uint32_t)d}, (uint32_t)sc, (size_t)(x + d + sc + fixed)};
    return true;
}

// The cheapest cut by estimate: rounds of the CTAs that an SM holds at once
// (two), at 3 us each, and the bytes at the rate of memory, those of a span
// that begins or ends inside a 32-byte sector counted with the whole sector.
static GnHeld held_plan(const GnCall &c, int sms, bool keep) {
    GnHeld best{0, 0, 0, 0, {0, 0}, 0, 0};
    double least = 0;
    const int es = bytes_of(c.dt);
    for (int K = 1; K <= c.G; ++K) {
        if (c.G % K != 0) continue;
        for (int n = 1; n <= kHeldCtas; n *= 2) {
            GnHeld h;
            if ((n > 1 && (c.S + n - 1) / n * (n - 1) >= c.S) || !held_cut(c, K, n, keep, h)) continue;
            const double row = (double)h.W * es, sectors = K == c.G || (h.W * es) % 32 == 0 ? row : row + 32;
            const double bytes = (double)c.B * c.S * c.C * es * (c.backward ? 3 : 2) * (sectors / row) * (row < 128 && K < c.G ? 1.25 : 1.0);
            // clusters of 16 leave SMs without a CTA where a GPU's groups of SMs are no multiple of 8
            const double ctas = (double)c.B * (c.G / K) * n, places = 2.0 * sms * (n == 16 ? 0.73 : n == 8 ? 0.94 : 1.0);
            const double rounds = std::ceil(ctas / places);
            const double share = ctas < sms ? sms / ctas : 1.0;  // SMs without a CTA
            const double cost = 3.0 * rounds + (n > 1 ? 0.5 : 0.0) + bytes * share / 6.7e6;
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

static int gn_threads(bool backward) { return backward ? 256 : 512; }

static GnPlan gn_plan(const GnCall &c, int sms) {
    GnPlan p;
    const int es = (c.dt & ~RMSNORM_WEIGHT_F32) == RMSNORM_F32 ? 4 : 2, E = c.wide ? 16 / es : 1;
    const int64_t CC = c.C / E;
    p.threads = gn_threads(c.backward);
    const int64_t cols = CC < p.threads ? CC : p.threads, lanes = p.threads / cols;
    // samples whose rows the L2 holds between the two passes over them
    const int64_t sample = c.S * c.C * es * (c.backward ? 2 : 1);
    int64_t batch = sample > 0 ? (int64_t)(48 << 20) / sample : c.B;
    p.batch = (int)(batch < 1 ? 1 : batch > c.B ? c.B : batch > 65535 ? 65535 : batch);
    // about four CTAs' worth of threads an SM; whole batches of rows a lane, 64 at most
    // (a lane's sums stay short) unless the chunks of a sample became more than 512
    const int64_t ctas = (int64_t)sms * (2048 / p.threads);
    int64_t per = (c.S * p.batch + ctas - 1) / ctas;
    int64_t k = (per + lanes - 1) / lanes;
    k = k > kGnBatch ? (k + kGnBatch - 1) / kGnBatch * kGnBatch : k;
    if (k > 64) k = 64;
    if (k < 1) k = 1;
    while ((c.S + k * lanes - 1) / (k * lanes) > 512) k *= 2;
    p.rows = (int)(k * lanes);
    p.chunks = (int)((c.S + p.rows - 1) / p.rows);
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    p.parts = 0;
    p.sums = up((size_t)c.B * p.chunks * 2 * (c.backward ? c.C : c.G) * sizeof(float));
    p.means = p.sums + (c.backward ? up((size_t)c.B * 2 * c.C * sizeof(float)) : 0);
    p.bytes = p.means + (c.backward ? up((size_t)c.B * c.G * sizeof(float2)) : 0);
    return p;
}

static bool gn_sizes(int64_t B, int64_t S, int64_t C, int64_t G, int act, int dt) {
    const int base = dt & ~RMSNORM_WEIGHT_F32;
    if (base != RMSNORM_F32 && base != RMSNORM_BF16 && base != RMSNORM_F16) return false;
    if (B < 0 || S < 0 || C < 1 || C > RMSNORM_MAX_N || G < 1 || C % G != 0) return false;
    if (B > 0x7fffffffLL || S > 0x7fffffffLL) return false;
    if (B > 0 && S > INT64_MAX / 8 / C / B) return false;
    return act >= kActNone && act <= kActGelu;
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
    p.magic = g.cg == 1 ? 0u : (uint32_t)(((1ull << 32) + g.cg - 1) / g.cg);
    p.status = status;
    const void *k = gn_held(base, c.backward, c.wide, c.act, c.backward ? c.kept : g.codes != nullptr);
    if (h.ctas > 8) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return head_cuda_fail((int)e);
    }
    void *args[] = {&p};
    const int64_t grid = c.B * p.spans * h.ctas;
    int e = launch(k, (unsigned)grid, 1, kHeldThreads, h.smem, args, s, (unsigned)h.ctas);
    if (e == 0 && c.backward && (dgamma || dbeta)) {
        const bool f32 = base == RMSNORM_F32 || g.w32;
        auto *fin = f32 ? launch_dw_finalize_f32 : base == RMSNORM_BF16 ? launch_dw_finalize_bf16 : launch_dw_finalize_f16;
        e = fin(g.parts, (int)(c.B * h.ctas), (int)(2 * c.C), dgamma, dbeta, (int)c.C, 0, s, false, sms);
    }
    return e == 0 ? RMSNORM_SUCCESS : head_cuda_fail(e);
}

static rmsnorm_status_t gn_run(GnParams &p, const GnCall &c, const GnPlan &plan, void *dgamma, void *dbeta, int sms,
                               cudaStream_t s) {
    const int base = c.dt & ~RMSNORM_WEIGHT_F32;
    const int E = c.wide ? (base == RMSNORM_F32 ? 4 : 8) : 1;
    const size_t stat = (size_t)p.G * sizeof(float2);
    void *args[] = {&p};
    int e = 0;
    const bool keep = !c.backward && p.codes;
    for (int64_t b0 = 0; b0 < c.B && e == 0; b0 += plan.batch) {
        p.b0 = (int)b0;
        const unsigned nb = (unsigned)(c.B - b0 < plan.batch ? c.B - b0 : plan.batch);
        if (!c.backward) {
            e = launch(gn_kernel(kGnStats, base, c.wide, 0, false), plan.chunks, nb, plan.threads,
                       2 * sizeof(float) * plan.threads * E + stat, args, s);
            if (e == 0) e = launch(gn_kernel(kGnApply, base, c.wide, c.act, keep), plan.chunks, nb, plan.threads, stat, args, s);
        } else {
            e = launch(gn_kernel(kGnBwdSums, base, c.wide, c.act, c.kept), plan.chunks, nb, plan.threads,
                       2 * sizeof(float) * plan.threads * E, args, s);
            int gpc = 1;
            while ((p.G + gpc - 1) / gpc > 4 * sms) gpc *= 2;
            void *rargs[] = {&p, &gpc};
            if (e == 0)
                e = launch(gn_kernel(kGnBwdReduce, base, c.wide, 0, false), (unsigned)((p.G + gpc - 1) / gpc), nb,
                           kGnReduceThreads, 0, rargs, s);
            if (e == 0) e = launch(gn_kernel(kGnBwdApply, base, c.wide, c.act, c.kept), plan.chunks, nb, plan.threads, 0, args, s);
        }
    }
    if (e == 0 && c.backward && (dgamma || dbeta)) {
        const bool f32 = base == RMSNORM_F32 || p.w32;
        auto *fin = f32 ? launch_dw_finalize_f32 : base == RMSNORM_BF16 ? launch_dw_finalize_bf16 : launch_dw_finalize_f16;
        e = fin(p.sums, (int)c.B, (int)(2 * c.C), dgamma, dbeta, (int)c.C, 0, s, false, sms);
    }
    return e == 0 ? RMSNORM_SUCCESS : head_cuda_fail(e);
}

static size_t gn_workspace(int64_t B, int64_t S, int64_t C, int64_t G, int dt, bool backward) {
    int sms = 0;
    if (!gn_sizes(B, S, C, G, 0, dt) || B == 0 || S == 0 || current_device(&sms, nullptr) != 0) return 0;
    size_t most = 0;
    for (int wide = 0; wide < 2; ++wide) {
        if (wide && C % (((dt & ~RMSNORM_WEIGHT_F32) == RMSNORM_F32) ? 4 : 8) != 0) continue;
        for (int kept = 0; kept < (backward ? 2 : 1); ++kept) {
            const GnCall c{B, S, C, (int)G, 0, dt, backward, kept != 0, wide != 0};
            const GnHeld h = held_plan(c, sms, false);
            if (h.ctas)
                most = backward ? std::max(most, held_bytes(c, h)) : most;
            else
                most = std::max(most, gn_plan(c, sms).bytes);
        }
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
    int sms = 0, *status = nullptr;
    const int e = current_device(&sms, &status);
    if (e != 0) return head_cuda_fail(e);
    GnCall c{B, S, C, (int)G, act, dt, false, false, C % (16 / es) == 0 && on(x, 16) && on(y, 16)};
    const GnPlan plan = gn_plan(c, sms);
    GnParams p;
    std::memset(&p, 0, sizeof p);
    p.x = x, p.gamma = gamma, p.beta = beta, p.out = y, p.mean = mean, p.rstd = rstd;
    p.S = S, p.B = (int)B, p.C = (int)C, p.G = (int)G, p.cg = (int)(C / G), p.rows = plan.rows, p.chunks = plan.chunks;
    p.act = act, p.w32 = (dt & RMSNORM_WEIGHT_F32) || base == RMSNORM_F32, p.eps = eps;
    // the codes in the same pass where rows are whole blocks of chunks
    const bool fused = codes && c.wide && C % kBlock8 == 0 && on(codes, 8);
    if (fused) p.codes = static_cast<uint8_t *>(codes), p.scales = scales;
    if (codes && !fused) {  // first: y may be x
        const rmsnorm_status_t st = ckpt8_pack(x, codes, scales, B * S, C, (rmsnorm_dtype_t)base, stream);
        if (st != RMSNORM_SUCCESS) return st;
    }
    const GnHeld h = held_plan(c, sms, fused);
    if (h.ctas) return gn_run_held(p, c, h, nullptr, nullptr, sms, status, s);
    return with_workspace(workspace, workspace_bytes, plan.bytes, s, [&](char *w) {
        p.parts = reinterpret_cast<float *>(w + plan.parts);
        return gn_run(p, c, plan, nullptr, nullptr, sms, s);
    });
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
    int sms = 0, *status = nullptr;
    const int e = current_device(&sms, &status);
    if (e != 0) return head_cuda_fail(e);
    GnCall c{B, S, C, (int)G, act, dt, true, codes != nullptr,
             C % (16 / es) == 0 && on(dy, 16) && on(dx, 16) && on(x, 16) && on(codes, 8)};
    const GnPlan plan = gn_plan(c, sms);
    GnParams p;
    std::memset(&p, 0, sizeof p);
    p.x = x, p.dy = dy, p.codes_in = static_cast<const uint8_t *>(codes), p.scales_in = scales;
    p.gamma = gamma, p.beta = beta, p.out = dx, p.mean = const_cast<float *>(mean), p.rstd = const_cast<float *>(rstd);
    p.S = S, p.B = (int)B, p.C = (int)C, p.G = (int)G, p.cg = (int)(C / G), p.rows = plan.rows, p.chunks = plan.chunks;
    p.act = act, p.w32 = (dt & RMSNORM_WEIGHT_F32) || base == RMSNORM_F32;
    const GnHeld h = held_plan(c, sms, false);
    return with_workspace(workspace, workspace_bytes, h.ctas ? held_bytes(c, h) : plan.bytes, s, [&](char *w) {
        p.parts = reinterpret_cast<float *>(w + plan.parts);
        if (h.ctas) return gn_run_held(p, c, h, dgamma, dbeta, sms, status, s);
        p.sums = reinterpret_cast<float *>(w + plan.sums);
        p.means = reinterpret_cast<float2 *>(w + plan.means);
        return gn_run(p, c, plan, dgamma, dbeta, sms, s);
    });
}

extern "C" size_t groupnorm_workspace_bytes(int64_t B, int64_t S, int64_t C, int64_t G, rmsnorm_dtype_t dt, int backward) {
    return gn_workspace(B, S, C, G, dt, backward != 0);
}
