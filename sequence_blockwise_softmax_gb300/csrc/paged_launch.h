// paged_launch.h -- the launches of paged attention's few-row form
// (attn_paged_tokens.cu) and few-key form (attn_paged_few.cu), shared with the
// entry point (attn_paged.cu), and the few-row form's rules on how a call is cut.
#pragma once
#include <cuda.h>

#include "ra_internal.h"
#include "ra_paged.cuh"

namespace ra {

constexpr int kPagedTokensRows = 32;        // most rows (new tokens x query heads) per key/value head
constexpr int kPagedTokensCtas = 2 * 152;   // two resident CTAs on each SM of a GB300
constexpr int kPagedMinRun = 4;             // chunks of a piece at least: one per warp
constexpr int kPagedWholeKeys = 1024;       // many pairs of at most so many keys: one CTA each, no pieces
constexpr int kPagedWholeSeqs = 512;        // of at most so many sequences

struct TokensLaunch {
    PagedSeqs seqs;
    const void *q, *k, *v;
    int64_t q_stride, page_stride;
    void *o;
    float *lse;
    bool o_bf16, whole_pairs;
    int d, ctas, cluster, row_blocks;
    float scale_log2;
    unsigned *status;
    unsigned long long *counters;   // kPagedTokensCtas
    float *part_o, *part_ml;    // [2 * ctas, rows up to 16 or 32, d], [.., 2]
};

// Whether every (sequence, key/value head) pair gets one CTA and is never cut:
// there are enough of them and they are short, and few enough sequences for each
// CTA to look at all of them: it reads their lengths, so a CTA to a pair costs the
// square of their number.  In us as pairs and as runs of all pairs, of 1-300 keys:
// 32 / 8 heads, d = 128: 160 sequences 33 and 50, 320: 67 and 82, 640: 145 and 114,
// 5120: 4330 and 770; 8 / 2 heads, d = 64: 12 and 20, 19 and 25, 36 and 34, 970 and
// 190.
inline bool paged_tokens_whole(int64_t pairs, int64_t keys, int64_t n_seqs) {
    return 2 * pairs > kPagedTokensCtas && keys <= kPagedWholeKeys && n_seqs <= kPagedWholeSeqs;
}

// The size of the cluster of CTAs that each pair gets, or 0.
// One sequence's 8 pairs, 32 / 8 heads, d = 128, in us as clusters of 2, 4, 8, 16
// and as pieces joined through the workspace: 100 keys 4.9, 4.9, 5.0, 6.2, 5.6; 700:
// 8.5, 6.4, 5.9, 6.6, 7.5; 2000: clusters of 8 and 16 7.4, 7.4, pieces 8.4; 4000: 10.3,
// 9.5, 10.8; 8000: 15.7, 13.0, 12.7.  8 sequences, 64 pairs, of 500-1000 keys: clusters
// of 2 and 4 10.1, 8.6, pieces 10.3; of 16-2000: 14.8, 11.5, 11.4; of 16-4000: 24.4,
// 17.7, 15.0.  19 sequences, 152 pairs, of 900-1000 keys: clusters of 2 12.4, pieces
// 20.9.  More CTAs than the GPU holds at once cost a second wave: 37 pairs of 1000
// keys as clusters of 8 11.6, 36 pairs 7.4.  At the limit of 576 keys a CTA, with 480,
// 512, 544 and 576, clusters against pieces: 32 pairs, d = 64, clusters of 8: 10.5 / 12.1,
// 10.5 / 12.2, 11.3 / 12.4, 11.3 / 12.8; d = 128: 12.6 / 14.2 to 13.6 / 15.3; 64 pairs, of 4:
// 12.5 / 14.8 to 13.6 / 16.0; 16 pairs, d = 64, of 8: 10.1 / 10.0 to 10.8 / 10.6; 8 pairs, of
// 16: 13.4 / 12.4 to 14.3 / 13.0.
inline int paged_tokens_cluster(int64_t pairs, int64_t keys) {
    // as many CTAs as have keys enough each
    int c = keys <= 128 ? 2 : keys <= (pairs <= 8 ? 256 : 768) ? 4 : keys <= (pairs <= 4 ? 512 : 2560) ? 8 : 16;
    // and as the GPU holds for all pairs
    while (c > 1 && pairs > (c == 16 ? 8 : c == 8 ? 36 : c == 4 ? 74 : 152)) c /= 2;
    // long sequences want all SMs, and even runs where their lengths differ
    const bool full = 10 * pairs * c >= 9 * kPagedTokensCtas;
    // (about 512 keys a CTA: a window of 4096 has sinks and new tokens beside it)
    return c > 1 && keys <= (int64_t)c * (full ? 1024 : 576) ? c : 0;
}

// CTAs for `pairs` (sequence, key/value head) pairs of up to `keys` keys: the
// grid, not the split, which the kernel takes from the lengths it finds.
inline int paged_tokens_ctas(int64_t pairs, int64_t keys, int64_t n_seqs) {
    if (const int cluster = paged_tokens_cluster(pairs, keys)) return (int)(pairs * cluster);
    if (paged_tokens_whole(pairs, keys, n_seqs)) return (int)pairs;
    // two CTAs to a pair at least, so that few pairs are cut on their own
    if (2 * pairs >= kPagedTokensCtas) return kPagedTokensCtas;
    const int64_t chunks = pairs * ((keys + kPagedChunk - 1) / kPagedChunk + 1);
    int64_t n = (chunks + kPagedMinRun - 1) / kPagedMinRun;
    if (n < 2 * pairs) n = 2 * pairs;
    return (int)(n < 1 ? 1 : n > kPagedTokensCtas ? kPagedTokensCtas : n);
}

ra_status launch_paged_tokens(const TokensLaunch &t, cudaStream_t stream);

constexpr int kPagedFewRows = 64;           // rows of a CTA
constexpr int kPagedFewRoom = 24;           // most 16-key chunks a CTA holds at a time

struct PagedFewLaunch {
    PagedSeqs seqs;                         // unit_tokens = kPagedFewRows / group
    const void *q, *k, *v;
    int64_t q_stride, page_stride;
    void *o;
    float *lse;
    bool o_bf16;
    int d, units;
    int64_t keys;                           // a row block's keys, as the call expects them
    float scale_log2;
    unsigned *status;
};

ra_status launch_paged_few(const PagedFewLaunch &t, cudaStream_t stream);

// Tree attention's tensor-core form (attn_tree.cuh).
constexpr int kTreeCtas = 152;              // one to each SM of a GB300
constexpr int kTreeMinRun = 2;              // tiles of a run at least

// The lists of tiles side by side: as many of the key/value heads as divide them, up to eight.
inline int tree_streams(int64_t H_kv) {
    int n = 8;
    while (H_kv % n) --n;
    return n;
}

// Whether a call of 17 to 32 rows to a pair runs there: with two row tiles a warp of the
// few-row form takes 2.3 us for 16 keys at d = 128 (1.2 at d = 64), which holds that form to 4.3
// TB/s.  8 nodes, in us, few-row form (in blocks of 16 rows where clusters hold them, see plan in
// attn_paged.cu) against runs, 32 / 8 heads, d = 128: one sequence of 1000 keys 8.9 / 13.7,
// 2000: 10.4 / 13.7, 3000: 12.2 / 13.8, 4000: 16 / 13.9, 16000: 45 / 24; 4 of 1000: 10.6 / 14.1, of
// 2000-4000: 22 / 23; 16 of 200-1000: 24 / 24, of 2000-4000: 74 / 45; 64 of 100-300: 36 / 35, of
// 1000-2000: 111 / 82; 8 / 2 heads, d = 64: one of 4000: 8.2 / 12.5, 8000: 13 / 13.5, 16000: 22 /
// 15.5; 16 of 2000-4000: 15.3 / 18.0, 64 of 1000-2000: 29 / 26.
inline bool tree_in_runs(int64_t pairs, int64_t keys, int d) {
    return keys * d > 400000 || (double)pairs * (double)(keys * d) > 1.6e7;
}

// Whether a unit may be longer than the kTreePart key tiles that are summed at a time: its table row can hold
// more, and its window, if any, sees more.
constexpr int kTreePart = 1024;
inline bool tree_in_parts(int64_t capacity, int64_t max_new, int64_t window, int64_t sinks) {
    const int64_t all = (capacity + 127) / 128;
    const int64_t seen = window > 0 ? (window + max_new) / 128 + sinks / 128 + 4 : all;
    return (seen < all ? seen : all) > kTreePart;
}

struct TreeLaunch {
    PagedSeqs seqs;                         // unit_tokens: tokens of a unit
    int64_t units;                          // at most
    int tile_tokens, page_box, two, ctas, streams, d;
    bool in_parts;
    void *o;
    float *lse;
    bool o_bf16;
    float scale_log2;
    unsigned *status;
    void *part_o, *part_ml, *cuts;          // 2 * ctas pieces of [256 rows, d] fp32, 16 bytes a row, 16 a CTA
};

ra_status launch_tree(const TreeLaunch &t, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                      cudaStream_t stream);

}  // namespace ra
