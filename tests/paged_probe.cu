// Test helper, not part of the library: runs the paged attention's own units,
// splits, walks and page needs (ra_paged.cuh) on the host and counts, for
// every new token and key, how often the kernel lets the pair through.
#include "ra_paged.cuh"

extern "C" {

// cnt[t * cap + key], cap = max_pages * page.  loaded[s * max_pages + i]: page
// i of sequence s is read.  Returns 0, or what went wrong.
int ra_test_paged(const int *seq_lens, const int *cu_q, int n_seqs, int T, int max_pages, int page, int H, int Hkv,
                  int unit_tokens, int max_new, int window, int sinks, int num_splits, int tail_share, int *cnt,
                  int *loaded, int *parts_seen) {
    ra::PagedSeqs q{};
    q.seq_lens = seq_lens;
    q.cu_q = cu_q;
    q.n_seqs = n_seqs;
    q.T = T;
    q.max_pages = max_pages;
    q.page = page;
    q.n_pages = 1;
    q.H = H;
    q.Hkv = Hkv;
    q.group = H / Hkv;
    q.unit_tokens = unit_tokens;
    q.max_new = max_new < T ? max_new : T;
    q.window = window;
    q.sinks = sinks;
    q.num_splits = num_splits;
    q.tail_share = tail_share;
    const size_t cap = (size_t)max_pages * page;
    const int box = page < 128 ? page : 128;
    const int64_t units = ra::paged_units(T, n_seqs, unit_tokens);
    for (int u = 0; u < units; ++u) {
        const int s = ra::paged_find_seq(q, u);
        const ra::PagedUnit pu = ra::paged_unit(q, s, u - ra::paged_first_unit(q, s));
        if (pu.n <= 0) continue;
        if (pu.t0 < 0 || pu.t0 + pu.n > T) return 1;
        if (pu.n * q.group > ra::paged_unit_rows(q)) return 2;
        const ra::RangeWalk whole = ra::paged_walk(q, pu);
        const int parts = ra::paged_split_count(q, whole.end), per = ra::paged_split_tiles(q, whole.end);
        if (parts < 1 || parts > num_splits) return 3;
        if (parts > *parts_seen) *parts_seen = parts;
        const ra::RowKeys first = ra::paged_row(q, pu.p0);
        int visited = 0;
        for (int part = 0; part < num_splits; ++part) {
            if (part >= parts) continue;
            ra::RangeWalk w = whole;
            if (num_splits > 1) {
                w.i = part * per;
                w.end = w.end < w.i + per ? w.end : w.i + per;
                if (whole.end > 0 && w.end <= w.i) return 4;
            }
            for (w.start_step(); w.valid(); w.next(), ++visited) {
                if (w.tile < 0) return 5;
                for (int k0 = w.tile * 128; k0 < w.tile * 128 + 128; k0 += box) {
                    const bool need = ra::paged_needed(first, pu.p0 + pu.n, pu.len, k0, box);
                    if (need && (size_t)k0 / page >= (size_t)max_pages) return 6;
                    if (need) loaded[(size_t)s * max_pages + k0 / page] = 1;
                    for (int i = 0; i < pu.n; ++i) {
                        const ra::RowKeys r = ra::paged_row(q, pu.p0 + i);
                        for (int k = k0; k < k0 + box; ++k)
                            if ((k >= r.lo && k < r.hi) || (k >= r.slo && k < r.shi)) {
                                if (!need || (size_t)k >= cap) return 7;
                                ++cnt[(size_t)(pu.t0 + i) * cap + k];
                            }
                    }
                }
            }
        }
        if (visited != whole.end) return 8;
    }
    return 0;
}

// The same for the few-row form's chunks.
int ra_test_paged_chunks(const int *seq_lens, const int *cu_q, int n_seqs, int T, int max_pages, int page, int max_new,
                         int window, int sinks, int *cnt) {
    ra::PagedSeqs q{};
    q.seq_lens = seq_lens;
    q.cu_q = cu_q;
    q.n_seqs = n_seqs;
    q.T = T;
    q.max_pages = max_pages;
    q.page = page;
    q.H = q.Hkv = q.group = 1;
    q.max_new = q.unit_tokens = max_new;
    q.window = window;
    q.sinks = sinks;
    const size_t cap = (size_t)max_pages * page;
    for (int s = 0; s < n_seqs; ++s) {
        const ra::PagedChunks l = ra::paged_chunks(q, s);
        if ((l.n > 0) != (l.count > 0)) return 1;
        if (l.n > 0 && (l.t0 < 0 || l.t0 + l.n > T)) return 2;
        for (int c = 0; c < l.count; ++c) {
            const int k0 = ra::paged_chunk_key(l, c);
            if (k0 < 0 || k0 % ra::kPagedChunk) return 3;
            if (c > 0 && k0 <= ra::paged_chunk_key(l, c - 1)) return 4;
            for (int i = 0; i < l.n; ++i) {
                const ra::RowKeys r = ra::paged_row(q, l.p0 + i);
                for (int k = k0; k < k0 + ra::kPagedChunk; ++k)
                    if ((k >= r.lo && k < r.hi) || (k >= r.slo && k < r.shi)) {
                        if (k >= l.len || (size_t)k >= cap) return 5;
                        ++cnt[(size_t)(l.t0 + i) * cap + k];
                    }
            }
        }
    }
    return 0;
}
}
