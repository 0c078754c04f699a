// ckpt8.cu -- entry points of rows kept in 8 bits, of the norm that keeps them
// and of embedding rows (declared in include/rmsnorm.h).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "embed.cuh"
#include "rows_kernels.cuh"
#include "train_rows.h"

namespace rmsn {

static const void *other_kernel(int which, int base) {
    return base == RMSNORM_BF16 ? rows_other_bf16(which) : base == RMSNORM_F16 ? rows_other_f16(which) : rows_other_f32(which);
}
static RowKernels fwd_kernel(int base, int src, int N, bool wide) {
    return base == RMSNORM_BF16  ? rows_fwd_bf16(src, N, wide)
           : base == RMSNORM_F16 ? rows_fwd_f16(src, N, wide)
                                 : rows_fwd_f32(src, N, wide);
}
static RowKernels bwd_kernel(int base, bool fused, int N, bool wide) {
    return base == RMSNORM_BF16  ? rows_bwd_bf16(fused, N, wide)
           : base == RMSNORM_F16 ? rows_bwd_f16(fused, N, wide)
                                 : rows_bwd_f32(fused, N, wide);
}

static bool matrix(int64_t M, int64_t N, int dt) {
    return known_dtype(dt) && M >= 0 && M <= 0x7fffffffLL && N >= 1 && N <= RMSNORM_MAX_N;
}
static bool scalars(float eps, float offset) { return std::isfinite(eps) && std::isfinite(offset) && eps >= 0.f; }

// A forward over rows: of the vectorised kernels where rows are whole 16-byte
// chunks on 16-byte boundaries, else of the one that takes any.
static rmsnorm_status_t run_fwd(RowsParams &p, int src, int dt, bool aligned, cudaStream_t s) {
    const int base = base_of(dt), E = 16 / bytes_of(dt);
    const bool wide = aligned && p.N % E == 0;
    const RowKernels k = fwd_kernel(base, src, p.N, wide);
    const int teams = k.tpr == 0 || k.tpr >= 256 ? 1 : 256 / k.tpr;
    void *args[] = {&p};
    const int e = launch(k.fwd, (unsigned)((p.M + (int64_t)teams - 1) / teams), 1, k.tpr > 256 ? k.tpr : 256, 0, args, s);
    return e == 0 ? RMSNORM_SUCCESS : head_cuda_fail(e);
}

// ---------------------------------------------------------------- backward --

struct BwdPlan {
    RowKernels k;
    int rows, depth, grid, threads;  // rows a stage, stages
    size_t smem, bytes;              // shared memory, workspace
    int dw_rows, dw_parts;           // rows of any length: the cut of dw's kernel
};

constexpr int kStageTarget = 16 * 1024;   // bytes a stage holds at least, where there are rows enough
constexpr int kBwdSmem = 110 * 1024;      // of a CTA: two an SM
constexpr int kBwdSmemWide = 220 * 1024;  // of a CTA of 512 threads: one an SM

static bool bwd_plan(int64_t M, int64_t N, int dt, bool fused, bool wide, int sms, BwdPlan &b) {
    const int es = bytes_of(dt), E = 16 / es;
    b.k = bwd_kernel(base_of(dt), fused, (int)N, wide && N % E == 0);
    b.dw_rows = b.dw_parts = 0;
    if (b.k.tpr == 0) {
        b.threads = 256, b.rows = b.depth = 0, b.smem = 0, b.grid = (int)M;
        const int64_t strips = (N + 255) / 256, want = (8 * (int64_t)sms + strips - 1) / strips;
        b.dw_rows = (int)std::max<int64_t>((M + want - 1) / want, 16);
        b.dw_parts = (int)((M + b.dw_rows - 1) / b.dw_rows);
        b.bytes = ((size_t)b.dw_parts * N * 4 + 255) / 256 * 256;
        return true;
    }
    if (b.k.r == 0) {  // value by value
        b.threads = 256, b.rows = b.depth = 0;
        const int teams = b.threads / b.k.tpr;
        b.smem = teams > 1 ? (size_t)N * 4 : 0;
        b.grid = (int)std::min<int64_t>((M + teams - 1) / teams, (int64_t)4 * sms);
        b.bytes = ((size_t)b.grid * N * 4 + 255) / 256 * 256;
        return true;
    }
    const int consumers = bwd_consumers(b.k.tpr);
    b.threads = consumers + 32;
    const int teams = consumers / b.k.tpr, an_sm = b.k.tpr > 256 ? 1 : 2;
    const size_t room = an_sm == 1 ? kBwdSmemWide : kBwdSmem;
    // whole turns of the teams, more of them where rows are short, fewer where
    // there would not be a stage for every CTA
    int turns = 1;
    while (turns < 64 && StageLayout(teams * b.k.r * turns, (int)N, es, fused).bytes < kStageTarget &&
           M >= (int64_t)teams * b.k.r * turns * 2 * an_sm * sms)
        turns *= 2;
    b.rows = teams * b.k.r * turns;
    const size_t stage = StageLayout(b.rows, (int)N, es, fused).bytes;
    b.depth = (int)std::min<size_t>(kStagesMost, room / stage);
    if (b.depth < 2) return false;
    b.smem = std::max((size_t)b.depth * stage, teams > 1 ? (size_t)N * 4 : 0);
    const int64_t blocks = (M + b.rows - 1) / b.rows;
    b.grid = (int)std::min<int64_t>(blocks, (int64_t)an_sm * sms);
    b.bytes = ((size_t)b.grid * N * 4 + 255) / 256 * 256;
    return true;
}

static rmsnorm_status_t norm_bwd(const void *dy, const void *dres, const void *codes, const uint8_t *scales, const void *w,
                                 const float *rstd, void *dx, void *dw, void *workspace, size_t workspace_bytes, int64_t M,
                                 int64_t N, int dt, float offset, cudaStream_t s) {
    const int base = base_of(dt), es = bytes_of(dt), wb = weight_bytes(dt);
    int sms = 0, *status = nullptr;
    int e = current_device(&sms, &status);
    if (e != 0) return head_cuda_fail(e);
    const bool wide = on(dy, 16) && on(dx, 16) && on(dres, 16) && on(w, 16) && on(codes, 16 / es);
    BwdPlan b;
    if (!bwd_plan(M, N, dt, dres != nullptr, wide, sms, b) && !bwd_plan(M, N, dt, dres != nullptr, false, sms, b))
        return RMSNORM_ERR_UNSUPPORTED;
    RowsBwdParams p;
    std::memset(&p, 0, sizeof p);
    p.dy = dy, p.dres = dres, p.w = w, p.codes = static_cast<const uint8_t *>(codes), p.scales = scales, p.rstd = rstd;
    p.dx = dx, p.M = (int)M, p.N = (int)N, p.w32 = wb == 4, p.stage_rows = b.rows, p.depth = b.depth, p.offset = offset;
    p.status = status;
    void *args[] = {&p};
    auto run = [&](char *ws) {
        p.ws = reinterpret_cast<float *>(ws);
        int le = 0;
        if (b.k.tpr == 0 && ws) {
            void *dargs[] = {&p, &b.dw_rows};
            le = launch(other_kernel(kDwAny, base), (unsigned)((N + 255) / 256), (unsigned)b.dw_parts, 256, 0, dargs, s);
        }
        if (le == 0) le = launch(b.k.fwd, (unsigned)b.grid, 1, b.threads, b.smem, args, s, b.k.r ? 1 : 0);
        if (le == 0 && ws) {
            auto *fin = wb == 4 ? launch_dw_finalize_f32 : base == RMSNORM_BF16 ? launch_dw_finalize_bf16 : launch_dw_finalize_f16;
            le = fin(p.ws, b.k.tpr ? b.grid : b.dw_parts, (int)N, dw, nullptr, (int)N, 0, s, false, sms);
        }
        return le == 0 ? RMSNORM_SUCCESS : head_cuda_fail(le);
    };
    if (!w) return run(nullptr);
    return with_workspace(workspace, workspace_bytes, b.bytes, s, run);
}

// --------------------------------------------------------------- embedding --

static bool id_type(int bytes) { return bytes == 4 || bytes == 8; }

struct EmbedPlan {
    int ctas, share, bits, passes, tiles;  // the sort: CTAs of the cluster (0: launches over tiles)
    int piece, pieces, words;
    size_t keys, vals, keys2, vals2, counts, present, open, ends, parts, bytes;
};

static EmbedPlan embed_plan(int64_t T, int64_t rows, int64_t N) {
    EmbedPlan p;
    // tokens of a piece: a team adds them one batch after the other, so few tokens are cut finer
    p.piece = T * N <= (int64_t)kEmbedSmall ? 8 : kEmbedPiece;
    int bits = 0;
    while (bits < 32 && (rows >> bits) != 0) ++bits;  // keys 0 .. rows
    p.passes = (bits + kSortBits - 1) / kSortBits;
    p.bits = (bits + p.passes - 1) / p.passes;
    p.tiles = (int)((T + kSortTile - 1) / kSortTile);
    p.ctas = 0;
    p.share = 0;
    if (T <= (int64_t)kSortCluster * kSortTile) {
        // a CTA more for each 1024 tokens
        p.ctas = 1;
        while (p.ctas < kSortCluster && (int64_t)p.ctas * kSortThreads < T) p.ctas *= 2;
        p.share = (int)((T + p.ctas - 1) / p.ctas);
    }
    p.pieces = (int)((T + p.piece - 1) / p.piece);
    p.words = (int)((rows + 31) / 32);
    size_t at = 0;
    auto take = [&at](size_t n) {
        const size_t a = at;
        at += (n + 255) / 256 * 256;
        return a;
    };
    p.keys = take((size_t)T * 4);
    p.vals = take((size_t)T * 4);
    p.keys2 = p.vals2 = p.counts = 0;
    if (!p.ctas) {
        p.keys2 = take((size_t)T * 4);
        p.vals2 = take((size_t)T * 4);
        p.counts = take((size_t)kSortBins * (p.tiles + 1) * 4);
    }
    p.present = take((size_t)p.words * 4);
    p.open = take((size_t)(p.pieces + 1) * 8);
    p.ends = take((size_t)rows * 4);
    p.parts = take((size_t)p.pieces * 2 * N * 4);
    p.bytes = at;
    return p;
}

static int run_sort(const EmbedPlan &b, SortParams &p, char *w, int dtype, bool out32, bool wide, int sms, cudaStream_t s) {
    auto at = [w](size_t o) { return reinterpret_cast<uint32_t *>(w + o); };
    if (b.ctas) {
        p.keys = at(b.keys), p.vals = at(b.vals);
        // the other SMs clear the rows without a token meanwhile (whole clusters of CTAs, one an SM)
        const int clear = p.early > 0 ? std::max(1, (sms - b.ctas) / b.ctas) * b.ctas : 0;
        void *args[] = {&p, const_cast<int *>(&b.share)};
        return launch(embed_sort_kernel(dtype, out32, wide), (unsigned)(b.ctas + clear), 1, kSortThreads,
                      sort_shared() + std::max((size_t)b.share * 16, (size_t)kClearWords * 4), args, s, (unsigned)b.ctas);
    }
    cudaError_t e = cudaMemsetAsync(p.present, 0, (size_t)b.words * 4, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(p.open, 0, 4, s);
    if (e != cudaSuccess) return (int)e;
    p.counts = at(b.counts);
    int le = 0;
    for (int i = 0; i < b.passes && le == 0; ++i) {
        // the last pass ends in keys and vals
        const bool here = (b.passes - 1 - i) % 2 == 0;
        p.shift = i * b.bits;
        p.keys = at(here ? b.keys : b.keys2), p.vals = at(here ? b.vals : b.vals2);
        p.keys_in = i == 0 ? nullptr : at(here ? b.keys2 : b.keys);
        p.vals_in = i == 0 ? nullptr : at(here ? b.vals2 : b.vals);
        void *args[] = {&p};
        le = launch(sort_kernel(1), (unsigned)b.tiles, 1, kSortThreads, sort_shared(), args, s);
        if (le == 0) le = launch(sort_kernel(2), 1u << b.bits, 1, kSortThreads, 0, args, s);
        if (le == 0) le = launch(sort_kernel(3), (unsigned)b.tiles, 1, kSortThreads, sort_shared(), args, s);
    }
    return le;
}

}  // namespace rmsn

using namespace rmsn;

// ------------------------------------------------------------ entry points --

extern "C" rmsnorm_status_t ckpt8_pack(const void *x, void *codes, uint8_t *scales, int64_t M, int64_t N,
                                       rmsnorm_dtype_t dt, rmsnorm_stream_t stream) {
    if (!known_dtype(dt) || base_of(dt) != dt || M < 0 || N < 1 || N > RMSNORM_MAX_N || M > INT64_MAX / 8 / N) return RMSNORM_ERR_INVALID_ARG;
    if (M == 0) return RMSNORM_SUCCESS;
    const int es = bytes_of(dt), E = 16 / es;
    if (!x || !codes || !scales || !on(x, es)) return RMSNORM_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    int e;
    if (N % kBlock8 == 0 && on(x, 16) && on(codes, E)) {
        int64_t chunks = M * N / E;
        const int64_t ctas = (chunks + 256 * kPackChunks - 1) / (256 * kPackChunks);
        if (ctas > 0x7fffffffLL) return RMSNORM_ERR_INVALID_ARG;
        void *args[] = {&x, &codes, &scales, &chunks};
        e = launch(other_kernel(kPackBlocks, dt), (unsigned)ctas, 1, 256, 0, args, s);
    } else {
        int n = (int)N;
        const int64_t runs = ((N + kBlock8 - 1) / kBlock8 + kRun - 1) / kRun, ctas = (M * runs + 7) / 8;
        if (ctas > 0x7fffffffLL) return RMSNORM_ERR_INVALID_ARG;
        void *args[] = {&x, &codes, &scales, &M, &n};
        e = launch(other_kernel(kPackAny, dt), (unsigned)ctas, 1, 256, 0, args, s);
    }
    return e == 0 ? RMSNORM_SUCCESS : head_cuda_fail(e);
}

extern "C" rmsnorm_status_t ckpt8_unpack(const void *codes, const uint8_t *scales, void *x, int64_t M, int64_t N,
                                         rmsnorm_dtype_t dt, rmsnorm_stream_t stream) {
    if (!known_dtype(dt) || base_of(dt) != dt || M < 0 || N < 1 || N > RMSNORM_MAX_N || M > INT64_MAX / 8 / N) return RMSNORM_ERR_INVALID_ARG;
    if (M == 0) return RMSNORM_SUCCESS;
    const int es = bytes_of(dt), E = 16 / es;
    if (!x || !codes || !scales || !on(x, es)) return RMSNORM_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    int e;
    if (N % kBlock8 == 0 && on(x, 16) && on(codes, E)) {
        int64_t chunks = M * N / E;
        const int64_t ctas = (chunks + 256 * kPackChunks - 1) / (256 * kPackChunks);
        if (ctas > 0x7fffffffLL) return RMSNORM_ERR_INVALID_ARG;
        void *args[] = {&codes, &scales, &x, &chunks};
        e = launch(other_kernel(kUnpackBlocks, dt), (unsigned)ctas, 1, 256, 0, args, s);
    } else {
        int n = (int)N;
        const int64_t runs = ((N + kBlock8 - 1) / kBlock8 + kRun - 1) / kRun, ctas = (M * runs + 7) / 8;
        if (ctas > 0x7fffffffLL) return RMSNORM_ERR_INVALID_ARG;
        void *args[] = {&codes, &scales, &x, &M, &n};
        e = launch(other_kernel(kUnpackAny, dt), (unsigned)ctas, 1, 256, 0, args, s);
    }
    return e == 0 ? RMSNORM_SUCCESS : head_cuda_fail(e);
}

extern "C" rmsnorm_status_t rmsnorm_fwd_ckpt8(const void *x, const void *residual, const void *w, void *y,
                                              void *residual_out, float *rstd, void *codes, uint8_t *scales, int64_t M,
                                              int64_t N, rmsnorm_dtype_t dt, float eps, float offset,
                                              rmsnorm_stream_t stream) {
    if (!matrix(M, N, dt) || !scalars(eps, offset) || (residual == nullptr) != (residual_out == nullptr)) return RMSNORM_ERR_INVALID_ARG;
    if (M == 0) return RMSNORM_SUCCESS;
    const int es = bytes_of(dt);
    if (!x || !y || !rstd || !codes || !scales || !on(x, es) || !on(y, es) || !on(residual, es) || !on(residual_out, es) ||
        !on(rstd, 4) || !on(w, weight_bytes(dt)))
        return RMSNORM_ERR_INVALID_ARG;
    RowsParams p;
    std::memset(&p, 0, sizeof p);
    p.x = x, p.residual = residual, p.w = w, p.y = y, p.h = residual_out, p.rstd = rstd;
    p.codes = static_cast<uint8_t *>(codes), p.scales = scales;
    p.M = (int)M, p.N = (int)N, p.w32 = weight_bytes(dt) == 4, p.eps = eps, p.offset = offset;
    const bool aligned = on(x, 16) && on(y, 16) && on(residual, 16) && on(residual_out, 16) && on(w, 16) && on(codes, 16 / es);
    return run_fwd(p, residual ? kSrcAdd : kSrcPlain, dt, aligned, (cudaStream_t)stream);
}

extern "C" rmsnorm_status_t rmsnorm_bwd_ckpt8(const void *dy, const void *dresidual_out, const void *codes,
                                              const uint8_t *scales, const void *w, const float *rstd, void *dx, void *dw,
                                              void *workspace, size_t workspace_bytes, int64_t M, int64_t N,
                                              rmsnorm_dtype_t dt, float offset, rmsnorm_stream_t stream) {
    if (!matrix(M, N, dt) || !std::isfinite(offset) || (w == nullptr) != (dw == nullptr)) return RMSNORM_ERR_INVALID_ARG;
    const int es = bytes_of(dt), wb = weight_bytes(dt);
    if (!on(w, wb) || !on(dw, wb)) return RMSNORM_ERR_INVALID_ARG;
    if (M == 0) return zeros({{dw, (size_t)N * wb}}, (cudaStream_t)stream);
    if (!dy || !codes || !scales || !rstd || !dx || !on(dy, es) || !on(dresidual_out, es) || !on(dx, es) || !on(rstd, 4))
        return RMSNORM_ERR_INVALID_ARG;
    return norm_bwd(dy, dresidual_out, codes, scales, w, rstd, dx, dw, workspace, workspace_bytes, M, N, dt, offset, (cudaStream_t)stream);
}

extern "C" size_t rmsnorm_bwd_ckpt8_workspace_bytes(int64_t M, int64_t N, rmsnorm_dtype_t dt) {
    int sms = 0;
    if (!matrix(M, N, dt) || M == 0 || current_device(&sms, nullptr) != 0) return 0;
    size_t most = 0;
    for (int k = 0; k < 4; ++k) {
        BwdPlan b;
        if (bwd_plan(M, N, dt, k & 1, k & 2, sms, b)) most = std::max(most, b.bytes);
    }
    return most;
}

extern "C" rmsnorm_status_t rmsnorm_embed_fwd(const void *ids, const void *table, const void *w, void *y, void *h,
                                              float *rstd, int64_t T, int64_t N, int64_t rows, int id_bytes,
                                              rmsnorm_dtype_t dt, float scale, float eps, float offset,
                                              rmsnorm_stream_t stream) {
    if (!matrix(T, N, dt) || !scalars(eps, offset) || !std::isfinite(scale) || !id_type(id_bytes) || rows < 0) return RMSNORM_ERR_INVALID_ARG;
    if (T == 0) return RMSNORM_SUCCESS;
    const int es = bytes_of(dt);
    if (!ids || !on(ids, id_bytes) || (!table && rows > 0) || !y || !h || !rstd || !on(table, es) || !on(y, es) || !on(h, es) ||
        !on(rstd, 4) || !on(w, weight_bytes(dt)))
        return RMSNORM_ERR_INVALID_ARG;
    RowsParams p;
    std::memset(&p, 0, sizeof p);
    p.x = table, p.ids = ids, p.id_bytes = id_bytes, p.vocab = rows, p.w = w, p.y = y, p.h = h, p.rstd = rstd;
    p.M = (int)T, p.N = (int)N, p.w32 = weight_bytes(dt) == 4, p.scale = scale, p.eps = eps, p.offset = offset;
    return run_fwd(p, kSrcEmbed, dt, on(table, 16) && on(y, 16) && on(h, 16) && on(w, 16), (cudaStream_t)stream);
}

extern "C" rmsnorm_status_t embed_fwd(const void *ids, const void *table, void *h, int64_t T, int64_t N, int64_t rows,
                                      int id_bytes, rmsnorm_dtype_t dt, float scale, rmsnorm_stream_t stream) {
    if (!matrix(T, N, dt) || base_of(dt) != dt || !std::isfinite(scale) || !id_type(id_bytes) || rows < 0) return RMSNORM_ERR_INVALID_ARG;
    if (T == 0) return RMSNORM_SUCCESS;
    const int es = bytes_of(dt), E = 16 / es;
    if (!ids || !on(ids, id_bytes) || (!table && rows > 0) || !h || !on(table, es) || !on(h, es)) return RMSNORM_ERR_INVALID_ARG;
    RowsParams p;
    std::memset(&p, 0, sizeof p);
    p.x = table, p.ids = ids, p.id_bytes = id_bytes, p.vocab = rows, p.h = h, p.M = (int)T, p.N = (int)N, p.scale = scale;
    cudaStream_t s = (cudaStream_t)stream;
    if (N % E != 0 || !on(table, 16) || !on(h, 16)) return run_fwd(p, kSrcEmbed, dt, false, s);
    int tiles = (int)((N / E + 127) / 128);
    void *args[] = {&p, &tiles};
    const int64_t ctas = (T * tiles + 7) / 8;
    if (ctas > 0x7fffffffLL) return RMSNORM_ERR_INVALID_ARG;
    const int e = launch(other_kernel(kEmbedRows, dt), (unsigned)ctas, 1, 256, 0, args, s);
    return e == 0 ? RMSNORM_SUCCESS : head_cuda_fail(e);
}

extern "C" rmsnorm_status_t embed_bwd(const void *dh, const void *ids, void *dtable, void *workspace,
                                      size_t workspace_bytes, int64_t T, int64_t N, int64_t rows, int id_bytes,
                                      rmsnorm_dtype_t dt, float scale, int accumulate, rmsnorm_stream_t stream) {
    if (!matrix(T, N, dt) || !std::isfinite(scale) || !id_type(id_bytes) || rows < 0 || rows > 0x7ffffffeLL) return RMSNORM_ERR_INVALID_ARG;
    const int es = bytes_of(dt), ob = weight_bytes(dt), E = 16 / es;
    cudaStream_t s = (cudaStream_t)stream;
    if (rows == 0) return RMSNORM_SUCCESS;
    if (!dtable || !on(dtable, ob)) return RMSNORM_ERR_INVALID_ARG;
    if (T == 0) return accumulate ? RMSNORM_SUCCESS : zeros({{dtable, (size_t)rows * N * ob}}, s);
    if (!dh || !on(dh, es) || !ids || !on(ids, id_bytes)) return RMSNORM_ERR_INVALID_ARG;
    int sms = 0;
    int e = current_device(&sms, nullptr);
    if (e != 0) return head_cuda_fail(e);
    const EmbedPlan b = embed_plan(T, rows, N);
    const bool wide = N % E == 0 && on(dh, 16) && on(dtable, 16), out32 = ob == 4 && es == 2;
    const int C = (int)(wide ? N / E : N);
    EmbedSumParams p;
    std::memset(&p, 0, sizeof p);
    p.dh = dh, p.dtable = dtable, p.rows = rows, p.T = (int)T, p.N = (int)N, p.piece = b.piece, p.pieces = b.pieces, p.accumulate = accumulate != 0;
    p.scale = scale;
    p.team = 8;
    while (p.team < 256 && p.team < C) p.team *= 2;
    p.slices = (C + p.team - 1) / p.team;
    const int teams = 256 / p.team;
    const int64_t sums = ((int64_t)b.pieces * p.slices + teams - 1) / teams;
    // rows without a token: some cleared beside the sort where one cluster sorts, the others by these CTAs
    const int64_t early = accumulate || !b.ctas ? 0 : std::min<int64_t>(rows, kClearEarly / (N * ob) / 32 * 32);
    const int64_t clears = accumulate ? 0 : (rows - early + 31) / 32 * p.slices;
    p.early = early;
    if (sums + clears > 0x7fffffffLL) return RMSNORM_ERR_INVALID_ARG;
    p.sum_ctas = (int)sums;
    return with_workspace(workspace, workspace_bytes, b.bytes, s, [&](char *w) {
        SortParams q;
        std::memset(&q, 0, sizeof q);
        q.ids = ids, q.id_bytes = id_bytes, q.rows = rows, q.T = (int)T, q.bits = b.bits, q.passes = b.passes, q.tiles = b.tiles;
        q.words = b.words;
        q.dtable = dtable, q.N = (int)N, q.early = early;
        q.present = reinterpret_cast<uint32_t *>(w + b.present);
        q.open = reinterpret_cast<uint32_t *>(w + b.open);
        int le = run_sort(b, q, w, base_of(dt), out32, wide, sms, s);
        p.keys = reinterpret_cast<uint32_t *>(w + b.keys);
        p.vals = reinterpret_cast<uint32_t *>(w + b.vals);
        p.present = q.present, p.open = q.open, p.ends = reinterpret_cast<uint32_t *>(w + b.ends), p.parts = reinterpret_cast<float *>(w + b.parts);
        void *args[] = {&p};
        if (le == 0) le = launch(embed_sum_kernel(base_of(dt), out32, wide), (unsigned)(sums + clears), 1, 256, 0, args, s);
        if (le == 0 && b.pieces > 1)
            le = launch(embed_join_kernel(base_of(dt), out32, wide), (unsigned)std::min<int64_t>(8 * sms, (int64_t)b.pieces * ((C + kJoinChunks - 1) / kJoinChunks)), 1, 256, 0, args, s);
        return le == 0 ? RMSNORM_SUCCESS : head_cuda_fail(le);
    });
}

extern "C" size_t embed_bwd_workspace_bytes(int64_t T, int64_t N, int64_t rows) {
    if (T <= 0 || T > 0x7fffffffLL || N < 1 || N > RMSNORM_MAX_N || rows < 1 || rows > 0x7ffffffeLL) return 0;
    return embed_plan(T, rows, N).bytes;
}
