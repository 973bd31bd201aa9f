// Test helper, not part of the library: runs on the host what the tree forms of
// paged attention run (ra_paged.cuh): the tensor-core form's units, splits, walk
// and chains, and the few-row form's chunks and windows, counting for every new
// token and place of the cache how often the pair is let through.
#include "ra_paged.cuh"

namespace {

ra::PagedSeqs seqs(const int *seq_lens, const int *cu_q, const int *parents, int n_seqs, int T, int max_pages, int page,
                   int H, int max_new, int window, int sinks) {
    ra::PagedSeqs q{};
    q.seq_lens = seq_lens;
    q.cu_q = cu_q;
    q.parents = parents;
    q.n_seqs = n_seqs;
    q.T = T;
    q.max_pages = max_pages;
    q.page = page;
    q.n_pages = 1;
    q.H = H;
    q.Hkv = 1;
    q.group = H;
    q.max_new = max_new < T ? max_new : T;
    q.window = window;
    q.sinks = sinks;
    return q;
}

}  // namespace

extern "C" {

// cnt[t * cap + place], cap = max_pages * page.  Returns 0, or what went wrong.
int ra_test_tree_tiles(const int *seq_lens, const int *cu_q, const int *parents, int n_seqs, int T, int max_pages, int page,
                       int H, int unit_tokens, int max_new, int window, int sinks, int num_splits, int tail_share, int *cnt) {
    ra::PagedSeqs q = seqs(seq_lens, cu_q, parents, n_seqs, T, max_pages, page, H, max_new, window, sinks);
    q.unit_tokens = unit_tokens;
    q.num_splits = num_splits;
    q.tail_share = tail_share;
    const size_t cap = (size_t)max_pages * page;
    const int64_t units = ra::paged_units(T, n_seqs, unit_tokens);
    static short node_parent[ra::kTreeMost];
    for (int u = 0; u < units; ++u) {
        const int s = ra::paged_find_seq(q, u);
        const ra::PagedUnit pu = ra::paged_unit(q, s, u - ra::paged_first_unit(q, s));
        if (pu.n <= 0) continue;
        bool bad = false;
        if (pu.first + pu.n > ra::kTreeMost) return 1;
        for (int i = 0; i < pu.first + pu.n; ++i)
            node_parent[i] = (short)ra::tree_parent(parents, pu.t0 - pu.first, i, bad);
        const int before = pu.p0 - pu.first;
        const ra::RowKeys first = ra::paged_first_row(q, pu);
        const ra::TreeWalk whole = ra::tree_walk(ra::paged_walk(q, pu));
        const int parts = ra::paged_split_count(q, whole.end), per = ra::paged_split_tiles(q, whole.end);
        for (int part = 0; part < parts; ++part) {
            for (int i = 0; i < pu.n; ++i) {
                const int node = pu.first + i;
                int depth = 0;
                if (window > 0)
                    for (int p = node_parent[node]; p >= 0; p = node_parent[p]) ++depth;
                const ra::RowKeys r = ra::tree_row(q, before + depth, before);
                ra::TreeChain chain;
                chain.start(node, depth, before, window, sinks);
                ra::TreeWalk w = whole;
                if (num_splits > 1) {
                    w.i = part * per;
                    w.end = w.end < w.i + per ? w.end : w.i + per;
                }
                for (w.start_step(); w.valid(); w.next()) {
                    if (w.tile < 0) return 2;
                    uint32_t drafted[4] = {0, 0, 0, 0};
                    if (w.tile * 128 + 128 > before) chain.tile(node_parent, w.tile * 128 - before, drafted);
                    for (int c = 0; c < 128; ++c) {
                        const int k = w.tile * 128 + c;
                        const bool bit = (drafted[c >> 5] >> (c & 31)) & 1;
                        const bool old = (k >= r.lo && k < r.hi) || (k >= r.slo && k < r.shi);
                        if (bit && old) return 3;
                        if (!bit && !old) continue;
                        if (!ra::paged_needed(first, pu.p0 + pu.n, pu.len, k, 1) || (size_t)k >= cap) return 4;
                        ++cnt[(size_t)(pu.t0 + i) * cap + k];
                    }
                }
            }
        }
    }
    return 0;
}

// The few-row form: chunks of 16 keys, chains as 32 bits.
int ra_test_tree_chunks(const int *seq_lens, const int *cu_q, const int *parents, int n_seqs, int T, int max_pages, int page,
                        int max_new, int window, int sinks, int *cnt) {
    ra::PagedSeqs q = seqs(seq_lens, cu_q, parents, n_seqs, T, max_pages, page, 1, max_new, window, sinks);
    q.unit_tokens = q.max_new;
    if (q.max_new > 32) return 1;
    const size_t cap = (size_t)max_pages * page;
    for (int s = 0; s < n_seqs; ++s) {
        const ra::PagedChunks cl = ra::paged_chunks(q, s);
        if (cl.n <= 0) continue;
        bool bad = false;
        uint32_t chain[32];
        const ra::RowKeys f = ra::tree_row(q, cl.p0, cl.p0), l = ra::paged_row(q, cl.p0 + cl.n - 1);
        const int all_lo = l.lo, all_hi = f.hi, all_shi = f.shi > f.slo ? f.shi : 0;
        for (int i = 0; i < cl.n; ++i) {
            const int p = ra::tree_parent(parents, cl.t0, i, bad);
            chain[i] = (1u << i) | (p >= 0 ? chain[p] : 0u);
            int depth = -1;
            for (uint32_t x = chain[i]; x; x &= x - 1) ++depth;
            const uint32_t seen = window > 0 && depth >= window ? ra::tree_window(chain[i], window, sinks - cl.p0) : chain[i];
            const ra::RowKeys r = ra::tree_row(q, cl.p0 + depth, cl.p0);
            for (int c = 0; c < cl.count; ++c) {
                const int k0 = ra::paged_chunk_key(cl, c);
                const bool whole = (k0 >= all_lo && k0 + 16 <= all_hi) || k0 + 16 <= all_shi;
                for (int k = k0; k < k0 + 16; ++k) {
                    const int node = k - cl.p0;
                    const bool bit = node >= 0 && node < 32 && ((seen >> node) & 1);
                    const bool old = (k >= r.lo && k < r.hi) || (k >= r.slo && k < r.shi);
                    if (whole && !bit && !old) return 2;
                    if (bit && old) return 3;
                    if (!bit && !old) continue;
                    if ((size_t)k >= cap || k >= cl.len) return 4;
                    ++cnt[(size_t)(cl.t0 + i) * cap + k];
                }
            }
        }
    }
    return 0;
}

}  // extern "C"
