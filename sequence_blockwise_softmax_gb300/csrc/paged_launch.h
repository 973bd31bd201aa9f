// paged_launch.h -- the launches of paged attention's few-row form
// (attn_paged_tokens.cu) and few-key form (attn_paged_few.cu), shared with the
// entry point (attn_paged.cu).
#pragma once
#include "ra_internal.h"
#include "ra_paged.cuh"

namespace ra {

constexpr int kPagedTokensRows = 32;        // most rows (new tokens x query heads) per key/value head
constexpr int kPagedTokensCtas = 2 * 152;   // two resident CTAs on each SM of a GB300

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
// CTA to look at all of them.
bool paged_tokens_whole(int64_t pairs, int64_t keys, int64_t n_seqs);

// The size of the cluster of CTAs that each pair gets, or 0.
int paged_tokens_cluster(int64_t pairs, int64_t keys);

// CTAs for `pairs` (sequence, key/value head) pairs of up to `keys` keys: the
// grid, not the split, which the kernel takes from the lengths it finds.
int paged_tokens_ctas(int64_t pairs, int64_t keys, int64_t n_seqs);

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
