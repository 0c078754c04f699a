// embed.cuh -- the gradient of embedding rows by sorted tokens: parameters
// shared by its kernels and the host.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace rmsn {

constexpr int kEmbedPiece = 32;      // sorted tokens that one team sums at most
constexpr int kEmbedSmall = 8 << 20;  // values (of all tokens) up to which it is 8
constexpr int kSortThreads = 1024;
constexpr int kSortBits = 9;         // of an id, a pass at most
constexpr int kSortBins = 1 << kSortBits;
constexpr int kSortTile = 8192;      // tokens a CTA sorts
constexpr int kSortCluster = 8;      // CTAs that sort together in shared memory

struct SortParams {
    const void *ids;
    uint32_t *keys_in, *vals_in, *keys, *vals;  // a pass over several launches: from, to (keys_in NULL: from ids)
    uint32_t *counts;   // [kSortBins, tiles] and the bins' totals behind them
    uint32_t *present;  // one bit a row of the table: some token is its
    uint32_t *open;     // [0]: how many pieces end inside a run (set to 0 here)
    void *dtable;       // (one cluster) whose first rows without a token are set to zero here
    int64_t rows;       // of the table; the key of ids outside it
    int64_t early;      // rows that are cleared beside the sort (a multiple of 32, or all)
    int T, N, id_bytes, shift, bits, passes, tiles, words;
};

struct EmbedSumParams {
    const void *dh;
    void *dtable;
    const uint32_t *keys, *vals, *present;
    uint32_t *open;     // [0]: count; then pairs from [2]: a piece that ends inside a run, the run's row
    uint32_t *ends;     // [rows]: the piece where a row's run ends, for runs over several
    float *parts;       // [pieces, 2, N]: the sums of a piece's first row and of its last one, where they are not whole
    int64_t rows, early;
    int T, N, piece, pieces, team, accumulate;
    int sum_ctas, slices;  // CTAs that sum, column slices of a row
    float scale;
};

constexpr int kClearWords = 8192;    // bits of rows that a clearing CTA holds at once, in words
constexpr int kJoinChunks = 64, kJoinLanes = 4;  // chunks of a row that a CTA joins, threads a chunk
constexpr int64_t kClearEarly = 48 << 20;        // bytes of rows that are cleared beside the sort

const void *embed_sort_kernel(int dtype, bool out32, bool wide);  // a cluster's
const void *sort_kernel(int which);  // 1, 2, 3: a pass's count, scan, move
size_t sort_shared();                // bytes of shared memory, without the pairs
const void *embed_sum_kernel(int dtype, bool out32, bool wide);
const void *embed_join_kernel(int dtype, bool out32, bool wide);

}  // namespace rmsn
