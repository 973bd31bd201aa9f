// paged_launch.h -- the launches of paged attention's few-row form
// (attn_paged_tokens.cu) and few-key form (attn_paged_few.cu), shared with the
// entry point (attn_paged.cu), and the few-row form's rules on how a call is cut.
#pragma once
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
    int d, ctas, cluster;
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

}  // namespace ra
