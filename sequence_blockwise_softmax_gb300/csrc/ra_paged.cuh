// ra_paged.cuh -- which rows, keys and pages a unit of paged attention has.
//
// Plain integer arithmetic callable from host and device (tests/paged_probe.cu
// runs it on the CPU).  New tokens are ragged: sequence s has the rows
// [cu_q[s], cu_q[s + 1]) of q, and row i of its n stands at position
// seq_lens[s] - n + i.  The query heads of one key/value head are packed into
// the rows of a 128-row tile, token by token: row r is token r / group, head
// r % group, so one read of a key serves the whole group.
//
// The counts on the device may hold anything: every function here stays inside
// the tables, and clips lengths to what a table row can hold.
#pragma once
#include <cstdint>

#include "ra_window.cuh"

namespace ra {

struct PagedSeqs {
    const int *table;       // [n_seqs, max_pages]
    const int *seq_lens;    // [n_seqs], the new tokens among them
    const int *cu_q;        // [n_seqs + 1]
    int n_seqs, T;          // T: rows of q
    int max_pages, page, n_pages;
    int H, Hkv, group;      // group = H / Hkv
    int unit_tokens;        // tokens of a unit
    int max_new;            // no sequence has more new tokens; rows past that are not computed
    int window, sinks;      // window 0: none
    int num_splits;         // most parts a unit's keys are cut into
    int tail_share;         // 0, or 1024ths of the keys in the last, shorter part
    const int *parents;     // [T], trees of new tokens (see tree_parent), or null: one token after another
};

// A unit: tokens [t0, t0 + n) of q, at positions p0 .. p0 + n - 1 of sequence
// s, whose cache holds `len` tokens.
struct PagedUnit {
    int s, t0, n, p0, len;
    int first;              // the unit's tokens before it in its sequence
};

RA_HD int paged_bound(const PagedSeqs &q, int i) { return (int)clamp64(q.cu_q[i], 0, q.T); }

RA_HD int paged_len(const PagedSeqs &q, int s) {
    return (int)clamp64(q.seq_lens[s], 0, (int64_t)q.max_pages * q.page);
}

// Units are numbered so that a sequence is found by a search in cu_q alone:
// its first unit is start / unit_tokens + s, and ceil(n / unit_tokens) units
// fit before the next sequence's first.
RA_HD int64_t paged_units(int64_t T, int64_t n_seqs, int unit_tokens) { return T / unit_tokens + n_seqs; }
RA_HD int paged_first_unit(const PagedSeqs &q, int s) { return paged_bound(q, s) / q.unit_tokens + s; }

// The last sequence whose first unit is not past u.
RA_HD int paged_find_seq(const PagedSeqs &q, int u) {
    int lo = 0, hi = q.n_seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (paged_first_unit(q, mid) <= u) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Unit number `local` of sequence s, whose rows are [c0, c1); n <= 0 if it has none.
RA_HD PagedUnit paged_unit_of(const PagedSeqs &q, int s, int c0, int c1, int len, int local) {
    PagedUnit u;
    const int n_new = c1 - c0;
    const int n = n_new < q.max_new ? n_new : q.max_new;
    u.s = s;
    u.first = local * q.unit_tokens;
    u.t0 = c0 + u.first;
    u.n = n - u.first < q.unit_tokens ? n - u.first : q.unit_tokens;
    if (local < 0) u.n = 0;     // a unit before the first sequence's rows
    u.len = len;
    u.p0 = u.len - n_new + u.first;
    return u;
}
RA_HD PagedUnit paged_unit(const PagedSeqs &q, int s, int local) {
    return paged_unit_of(q, s, paged_bound(q, s), paged_bound(q, s + 1), paged_len(q, s), local);
}

// The keys of the token at position p (a negative position sees none).
RA_HD RowKeys paged_row(const PagedSeqs &q, int p) { return window_row_keys(0, p, q.window, q.sinks); }

// The keys that bound a unit's: its first row's, or with trees, whose rows all
// stand at the first new token's position or behind it, those of a row there.
RA_HD RowKeys paged_first_row(const PagedSeqs &q, const PagedUnit &u) {
    return paged_row(q, q.parents ? u.p0 - u.first : u.p0);
}

RA_HD RangeWalk paged_walk(const PagedSeqs &q, const PagedUnit &u) {
    return range_walk(paged_first_row(q, u), u.p0 + u.n);
}

// Whether sequence s breaks the call's bounds: more new tokens than max_new or
// than its length, or a length its table row cannot hold.
RA_HD bool paged_bad_counts(const PagedSeqs &q, int s) {
    const int n_new = paged_bound(q, s + 1) - paged_bound(q, s);
    return n_new > q.max_new || n_new > q.seq_lens[s] ||
           (int64_t)q.seq_lens[s] > (int64_t)q.max_pages * q.page;
}

// The most tokens a unit can hold, and its rows in the join's buffers.
RA_HD int paged_unit_rows(const PagedSeqs &q) {
    return (q.max_new < q.unit_tokens ? q.max_new : q.unit_tokens) * q.group;
}

// A unit's tiles are cut into at most num_splits parts of equal size, at least
// kSplitTiles tiles each: a part costs its CTA about 8 us and the join a read
// of its rows, a tile 1.35 us (1.0 at d = 64).  With tail_share (at most a part's equal
// share) the last part has that much and the others the rest.
constexpr int kSplitTiles = 6;
RA_HD int paged_split_tiles(const PagedSeqs &q, int tiles) {
    int ns = tiles / kSplitTiles;
    if (ns > q.num_splits) ns = q.num_splits;
    if (ns < 1) ns = 1;
    if (q.tail_share > 0 && ns > 1 && ns == q.num_splits) {
        const int tail = (int)((int64_t)tiles * q.tail_share >> 10);
        return (tiles - tail + ns - 2) / (ns - 1);
    }
    return (tiles + ns - 1) / ns;
}
RA_HD int paged_split_count(const PagedSeqs &q, int tiles) {
    const int per = paged_split_tiles(q, tiles);
    return per > 0 ? (tiles + per - 1) / per : 1;
}

// Whether the keys [k0, k0 + n) hold one that a row of the walk's unit sees:
// `first` is its first row's keys, last_hi one past its last row's position.
RA_HD bool paged_needed(const RowKeys &first, int last_hi, int len, int k0, int n) {
    if (k0 >= len) return false;
    return (k0 < last_hi && k0 + n > first.lo) || (k0 < first.shi && k0 + n > first.slo);
}

constexpr int kPagedChunk = 16;

// The few-row form (attn_paged_tokens.cu): the 16-key chunks of sequence s's keys that its new tokens (those of block number `block`) see, in order:
// n_sink chunks from 0 on, then chunks from m0 on.  A sequence with new tokens
// that see nothing keeps one (masked) chunk, so that its rows are written.
struct PagedChunks {
    int n_sink, m0, count;
    int t0, n, p0, len;      // its new tokens, their first position, its length
    int first;               // new tokens of the sequence before them
};
RA_HD PagedChunks paged_chunks(const PagedSeqs &q, int s, int block = 0) {
    PagedChunks c;
    const PagedUnit u = paged_unit(q, s, block);
    c.first = u.first;
    c.t0 = u.t0;
    c.n = u.n;
    c.p0 = u.p0;
    c.len = u.len;
    c.n_sink = c.m0 = c.count = 0;
    if (u.n <= 0) return c;
    const RowKeys first = paged_first_row(q, u);
    const int last = u.p0 + u.n;
    c.m0 = first.lo / kPagedChunk;
    const int m1 = (last + kPagedChunk - 1) / kPagedChunk;
    if (first.shi > first.slo) {
        const int s1 = (first.shi + kPagedChunk - 1) / kPagedChunk;
        c.n_sink = s1 < c.m0 ? s1 : c.m0;
    }
    c.count = c.n_sink + (m1 > c.m0 ? m1 - c.m0 : 0);
    if (c.count == 0) c.count = 1;
    return c;
}

// One sequence's share of a sum over all of them, which counts the sequences
// with chunks above bit 39 and their chunks but one below.  Up to 2^24 sequences
// of 2^39 chunks in all (a call's limits) stay inside its 64 bits.
constexpr int kPagedTallyBits = 39;
RA_HD uint64_t paged_tally(int chunks) {
    return chunks > 0 ? ((uint64_t)1 << kPagedTallyBits) + (uint64_t)(chunks - 1) : 0;
}
RA_HD int64_t paged_tally_seqs(uint64_t sum) { return (int64_t)(sum >> kPagedTallyBits); }
RA_HD int64_t paged_tally_chunks(uint64_t sum) {
    return (int64_t)(sum & (((uint64_t)1 << kPagedTallyBits) - 1)) + paged_tally_seqs(sum);
}

// The first key of chunk number c.
RA_HD int paged_chunk_key(const PagedChunks &l, int c) {
    return (c < l.n_sink ? c : l.m0 + (c - l.n_sink)) * kPagedChunk;
}

// Trees of new tokens.  Row i of a sequence follows row parents[cu[s] + i] < i
// of the same sequence, or with -1 the c = seq_lens[s] - n tokens before the
// new ones.  It lies at place c + i of the cache and stands at position c +
// depth, its depth the number of its ancestors; it sees the c tokens, its
// ancestors and itself, of which a window leaves those less than `window`
// positions away and the sinks.  A chain of ancestors has falling numbers and
// positions, so what a window leaves of it are its first `window` nodes from
// the row up, and as many at the other end as stand before the sinks' end.
constexpr int kTreeMost = 1024;     // new tokens of a sequence

// Row i's parent; what is none of -1 .. i - 1 counts as -1 and is `bad`.
RA_HD int tree_parent(const int *parents, int t0, int i, bool &bad) {
    const int p = parents[t0 + i];
    if (p >= -1 && p < i) return p;
    bad = true;
    return -1;
}

// What the row at position p sees of the c tokens before the new ones.
RA_HD RowKeys tree_row(const PagedSeqs &q, int p, int c) {
    RowKeys r = paged_row(q, p);
    if (r.hi > c) r.hi = c;
    if (r.shi > c) r.shi = c;
    return r;
}

// What a window leaves of a chain given as the bits of its nodes, of at most
// 32: the `window` highest, and the lowest `near` (nodes before the sinks' end).
RA_HD uint32_t tree_window(uint32_t chain, int window, int near) {
    int n = 0;
    for (uint32_t x = chain; x; x &= x - 1) ++n;
    uint32_t keep = 0;
    for (int i = 0; i < n - window; ++i) {
        const uint32_t low = chain & (0u - chain);
        chain ^= low;
        if (i < near) keep |= low;
    }
    return chain | keep;
}

// A row's chain walked up as its unit's key tiles go down.
struct TreeChain {
    int at, steps;      // the node next in turn (-1: none left), its distance from the row
    int window, far;    // nodes of a distance below `window` or above `far` are seen

    // row `node` with `depth` ancestors; window 0: none (depth is then not used)
    RA_HD void start(int node, int depth, int c, int win, int sinks) {
        at = node;
        steps = 0;
        window = win > 0 ? win : 0x7fffffff;
        far = win > 0 ? c + depth - sinks : 0x7fffffff;
    }
    // the seen nodes of [base, base + 128), bit i & 31 of word i >> 5 for node base + i
    template <class Parent>
    RA_HD void tile(const Parent *parents, int base, uint32_t (&word)[4]) {
        word[0] = word[1] = word[2] = word[3] = 0;
        while (at >= 0 && at >= base) {
            const int i = at - base;
            if (i < 128 && (steps < window || steps > far)) {
                const uint32_t bit = 1u << (i & 31);
                word[0] |= i < 32 ? bit : 0u;
                word[1] |= i >= 32 && i < 64 ? bit : 0u;
                word[2] |= i >= 64 && i < 96 ? bit : 0u;
                word[3] |= i >= 96 ? bit : 0u;
            }
            at = parents[at];
            ++steps;
        }
    }
};

// The key tiles of a unit of tree rows: the main ones from the last down, then
// the sinks'.
struct TreeWalk {
    int i, end, n_main, last, s0;
    int tile;

    RA_HD_STEP void seek() { tile = i < n_main ? last - i : s0 + (i - n_main); }
    RA_HD_STEP bool valid() const { return i < end; }
    RA_HD_STEP void next() {
        ++i;
        seek();
    }
};
RA_HD TreeWalk tree_walk(const RangeWalk &r) {
    TreeWalk w;
    w.i = r.i;
    w.end = r.end;
    w.n_main = r.end - r.n_sink;
    w.last = r.m0 + w.n_main - 1;
    w.s0 = r.s0;
    w.tile = 0;
    return w;
}

}  // namespace ra
