// Test helper, not part of the library: runs on the host what the tree forms of
// paged attention run (ra_paged.cuh, ra_tree.cuh): the tensor-core form's units,
// runs, walk and chains, and the few-row form's blocks, chunks and windows, counting
// for every new token and place of the cache how often the pair is let through.
#include <vector>

#include "ra_paged.cuh"
#include "ra_tree.cuh"

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

// cnt[(t * Hkv + head) * cap + place], cap = max_pages * page: `streams` lists of Hkv / streams
// heads, `runs` runs of each, of min_run places at least; two: the units have two Q tiles; tried: receives how often
// units were cut on their own.  Returns 0, or what went wrong.
int ra_test_tree_runs(const int *seq_lens, const int *cu_q, const int *parents, int n_seqs, int T, int max_pages, int page,
                      int group, int Hkv, int unit_tokens, int max_new, int window, int sinks, int streams, int runs,
                      int min_run, int two, int *tried, int *cnt) {
    ra::PagedSeqs q = seqs(seq_lens, cu_q, parents, n_seqs, T, max_pages, page, group * Hkv, max_new, window, sinks);
    q.Hkv = Hkv;
    q.group = group;
    q.unit_tokens = unit_tokens;
    const size_t cap = (size_t)max_pages * page;
    const int heads = Hkv / streams;
    static short node_parent[ra::kTreeMost];
    std::vector<int> stored((size_t)T * Hkv);       // how often a row's unit was begun
    for (int stream = 0; stream < streams; ++stream) {
        const int head0 = stream * heads;
        long long total = 0;
        for (int s = 0; s < n_seqs; ++s) total += ra::tree_head_cost(q, ra::tree_seq(q, s)) * heads;
        long long per = ra::tree_per(total, runs, min_run, two), units = 0;
        for (int s = 0; s < n_seqs; ++s) units += ra::tree_seq(q, s).blocks;
        const int pad = ra::tree_pad(units * heads, total, runs, per, two ? 1 : 2);
        if (pad > 1) {
            per = pad;
            total = 0;
            for (int s = 0; s < n_seqs; ++s) total += ra::tree_head_cost(q, ra::tree_seq(q, s), pad) * heads;
            if (total > runs * per) return 15;
            ++*tried;
        }
        struct {
            int more, run, t0, hk;
        } open{0, 0, 0, 0};        // the unit that the run before left, and in how many runs it goes on
        for (int run = 0; run < runs; ++run) {
            long long pos = run * per;
            const long long end = pos + per < total ? pos + per : total;
            if (pos >= total) break;
            long long off = pos;
            int s = 0;
            for (long long c; off >= (c = ra::tree_head_cost(q, ra::tree_seq(q, s), pad) * heads); ++s) off -= c;
            ra::TreeSeq seq = ra::tree_seq(q, s);
            ra::TreeSegment e = ra::tree_first_segment(q, seq, ra::tree_head_cost(q, seq, pad), head0, off, pos, end, per, run, pad);
            int cuts = 0;
            for (bool first_of_run = true;; first_of_run = false) {
                if (e.tiles < 0 || e.places < 1 || e.n < 1 || e.hk < head0 || e.hk >= head0 + heads) return 1;
                if (e.t0 < 0 || e.t0 + e.n > T || e.first + e.n > ra::kTreeMost) return 2;
                if (!first_of_run && (!e.begins || pad > 1)) return 3;
                if (e.tiles == 0 && e.i0 > 0) return 16;
                if (!e.begins) {
                    // the unit left open, until its note's last run
                    if (open.t0 != e.t0 || open.hk != e.hk || run > open.run + open.more) return 4;
                    if ((e.more > 0) != (run < open.run + open.more)) return 5;
                } else {
                    if (first_of_run && run > 0 && open.run + open.more >= run) return 6;
                    for (int i = 0; i < e.n; ++i) ++stored[(size_t)(e.t0 + i) * Hkv + e.hk];
                    if (!e.whole) {
                        open = {e.more, run, e.t0, e.hk};
                        if (++cuts > 1 || e.more < 1) return 7;
                    }
                }
                if (e.whole != (e.begins && e.more == 0)) return 8;
                bool bad = false;
                for (int i = 0; i < e.first + e.n; ++i)
                    node_parent[i] = (short)ra::tree_parent(parents, e.t0 - e.first, i, bad);
                const ra::RowKeys first = ra::paged_row(q, e.before);
                for (int i = 0; i < e.n; ++i) {
                    const int node = e.first + i;
                    int depth = 0;
                    if (window > 0)
                        for (int p = node_parent[node]; p >= 0; p = node_parent[p]) ++depth;
                    const ra::RowKeys r = ra::tree_row(q, e.before + depth, e.before);
                    if (r.hi != e.before && e.before >= 0) return 9;
                    ra::TreeChain chain;
                    chain.start(node, depth, e.before, window, sinks);
                    for (int j = 0; j < e.tiles; ++j) {
                        const int tile = ra::tree_tile(e, j);
                        if (tile < 0) return 10;
                        uint32_t drafted[4] = {0, 0, 0, 0};
                        if (tile * 128 + 128 > e.before) chain.tile(node_parent, tile * 128 - e.before, drafted);
                        for (int c = 0; c < 128; ++c) {
                            const int k = tile * 128 + c;
                            const bool bit = (drafted[c >> 5] >> (c & 31)) & 1;
                            // (as the kernel masks: the sinks from 0 up to shi)
                            const bool old = (k >= r.lo && k < e.before) || k < r.shi;
                            if (bit && old) return 11;
                            if (!bit && !old) continue;
                            if (!ra::paged_needed(first, e.before + e.first + e.n, e.len, k, 1) || (size_t)k >= cap) return 12;
                            ++cnt[((size_t)(e.t0 + i) * Hkv + e.hk) * cap + k];
                        }
                    }
                }
                pos += e.places;
                if (pos > end) return 13;
                if (pos == end) break;
                e = ra::tree_next_segment(q, seq, e, head0, heads, pos, end, per, run, pad);
            }
        }
    }
    for (int s = 0; s < n_seqs; ++s)
        for (int t = cu_q[s]; t < cu_q[s + 1] && t < cu_q[s] + max_new; ++t)
            for (int h = 0; h < Hkv; ++h)
                if (stored[(size_t)t * Hkv + h] != 1) return 14;
    return 0;
}

// The few-row form: chunks of 16 keys, chains as 32 bits.
int ra_test_tree_chunks(const int *seq_lens, const int *cu_q, const int *parents, int n_seqs, int T, int max_pages, int page,
                        int max_new, int window, int sinks, int block, int *cnt) {
    ra::PagedSeqs q = seqs(seq_lens, cu_q, parents, n_seqs, T, max_pages, page, 1, max_new, window, sinks);
    q.unit_tokens = block;
    const int blocks = (q.max_new + block - 1) / block;
    if (q.max_new > 32) return 1;
    const size_t cap = (size_t)max_pages * page;
    for (int v = 0; v < n_seqs * blocks; ++v) {
        const ra::PagedChunks cl = ra::paged_chunks(q, v / blocks, v % blocks);
        if (cl.n <= 0) continue;
        bool bad = false;
        uint32_t chain[32];
        const int before = cl.p0 - cl.first;
        const ra::RowKeys f = ra::tree_row(q, before, before), l = ra::paged_row(q, cl.p0 + cl.n - 1);
        const int all_lo = l.lo, all_hi = f.hi, all_shi = f.shi > f.slo ? f.shi : 0;
        for (int i = 0; i < cl.first + cl.n; ++i) {
            const int p = ra::tree_parent(parents, cl.t0 - cl.first, i, bad);
            chain[i] = (1u << i) | (p >= 0 ? chain[p] : 0u);
            if (i < cl.first) continue;
            int depth = -1;
            for (uint32_t x = chain[i]; x; x &= x - 1) ++depth;
            const uint32_t seen = window > 0 && depth >= window ? ra::tree_window(chain[i], window, sinks - before) : chain[i];
            const ra::RowKeys r = ra::tree_row(q, before + depth, before);
            for (int c = 0; c < cl.count; ++c) {
                const int k0 = ra::paged_chunk_key(cl, c);
                const bool whole = (k0 >= all_lo && k0 + 16 <= all_hi) || k0 + 16 <= all_shi;
                for (int k = k0; k < k0 + 16; ++k) {
                    const int node = k - before;
                    const bool bit = node >= 0 && node < 32 && ((seen >> node) & 1);
                    const bool old = (k >= r.lo && k < r.hi) || (k >= r.slo && k < r.shi);
                    if (whole && !bit && !old) return 2;
                    if (bit && old) return 3;
                    if (!bit && !old) continue;
                    if ((size_t)k >= cap || k >= cl.len) return 4;
                    ++cnt[(size_t)(cl.t0 + i - cl.first) * cap + k];
                }
            }
        }
    }
    return 0;
}

}  // extern "C"
