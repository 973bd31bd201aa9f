// ra_tree.cuh -- how tree attention's units of rows are cut into runs of key tiles.
//
// Plain integer arithmetic callable from host and device (tests/tree_probe.cu
// runs it on the CPU).  A list has the units of some key/value heads, sequence by
// sequence, head by head, block of rows by block, and each unit as many places
// as it has key tiles; a run is `per` places in a row.  A run that ends one unit and
// begins another pays for both ends (about 3.5 us), so where there are runs enough each
// unit is cut on its own: it then has places for whole runs, `pad` at a time (tree_pad).
// 60 nodes over 1100 keys, 32 / 8 heads, d = 128: 17.2 us cut anywhere, 14.7 so; 3
// sequences of 1500-3500: 25.2 and 21.8; for about 0.5 us where it changes nothing.
#pragma once
#include "ra_paged.cuh"

namespace ra {

// a / b for b > 0, a >= 0
RA_HD long long div_pos(long long a, long long b) {
    return (a | b) >> 32 ? a / b : (long long)((unsigned)a / (unsigned)b);
}
RA_HD int tree_max(int a, int b) { return a > b ? a : b; }

// A piece of a unit: `tiles` tiles of its walk from number i0 on (tiles < 0: the
// queue's end).  The walk's n_main, last and s0 are TreeWalk's.
struct __align__(16) TreeSegment {
    int tiles, i0, n_main, last, s0;
    int s, hk, t0, n, first;        // sequence, head, the unit's tokens (PagedUnit)
    int before, len;                // the sequence's tokens before the new ones, and in all
    int whole;                      // the piece is the unit
    int begins, more;               // in the CTA's run; how many runs it goes on through
    int places;                     // of the list
};
static_assert(sizeof(TreeSegment) == 64, "a quarter of a shared-memory line");

// Key tile number j of a segment (TreeWalk's order).
RA_HD int tree_tile(const TreeSegment &e, int j) {
    const int i = e.i0 + j;
    return i < e.n_main ? e.last - i : e.s0 + (i - e.n_main);
}

// A sequence as a run meets it: rows [c0, c1), len tokens in the cache, and the blocks
// (units of one head) of its rows.
struct TreeSeq {
    int s, c0, c1, len, blocks;
};
RA_HD TreeSeq tree_seq(const PagedSeqs &q, int s) {
    TreeSeq t;
    t.s = s;
    t.c0 = paged_bound(q, s);
    t.c1 = paged_bound(q, s + 1);
    t.len = paged_len(q, s);
    const int n = t.c1 - t.c0 < q.max_new ? t.c1 - t.c0 : q.max_new;
    t.blocks = n > 0 ? (n + q.unit_tokens - 1) / q.unit_tokens : 0;
    return t;
}
RA_HD PagedUnit tree_unit(const PagedSeqs &q, const TreeSeq &t, int b) {
    return paged_unit_of(q, t.s, t.c0, t.c1, t.len, b);
}
// Places of a unit of so many tiles; one that sees no key takes some all the
// same, so that its rows are written.
RA_HD int tree_places(int tiles, int pad) {
    const int n = tree_max(tiles, 1);
    return pad > 1 ? (n + pad - 1) / pad * pad : n;
}
RA_HD int tree_block_cost(const PagedSeqs &q, const TreeSeq &t, int b, int pad = 1) {
    return tree_places(paged_walk(q, tree_unit(q, t, b)).end, pad);
}
RA_HD long long tree_head_cost(const PagedSeqs &q, const TreeSeq &t, int pad = 1) {
    long long sum = 0;
    for (int b = 0; b < t.blocks; ++b) sum += tree_block_cost(q, t, b, pad);
    return sum;
}
// How long the pieces are when each unit is cut on its own: per, or `step` tiles more where that is
// little, as it takes that the runs suffice whatever the units' lengths; 1 where they do not or
// there is one unit.  (No division: this stands before a CTA's first load.)
RA_HD int tree_pad(long long units, long long total, int runs, long long per, int step) {
    if (units == 1 || units * 2 > runs || total > (1 << 28)) return 1;
    for (int k = 0; k < (per < 6 ? 1 : 2); ++k, per += step)
        if (total + units * (per - 1) < (runs + 1) * per) return (int)per;
    return 1;
}

// A run's places: an equal share of the list, and where two groups take a unit's tiles in turn 4
// instead of 3, which take as long (30 nodes over 5000 keys, 32 / 8 heads, d = 128: 16.6 us
// against 17.8; but 6 for 5 lose 2, of two sequences of up to 8000).
RA_HD long long tree_per(long long total, int runs, int least, bool two) {
    long long per = div_pos(total + runs - 1, runs);
    if (per < least) per = least;
    return !two && per == 3 ? 4 : per;
}

// The part of block b of a sequence from tile i0 of it on that lies in a run, whose places from
// `pos` on it takes.
RA_HD TreeSegment tree_segment(const PagedSeqs &q, const TreeSeq &t, int head, int b, int i0, long long pos, long long end,
                               long long per, int run, int pad = 1) {
    const PagedUnit u = tree_unit(q, t, b);
    const TreeWalk w = tree_walk(paged_walk(q, u));
    const int cost = tree_places(w.end, pad), i1 = cost < i0 + (end - pos) ? cost : (int)(i0 + (end - pos));
    TreeSegment e;
    e.places = i1 - i0;
    e.i0 = i0 < w.end ? i0 : w.end;
    e.tiles = (i1 < w.end ? i1 : w.end) - e.i0;
    e.n_main = w.n_main;
    e.last = w.last;
    e.s0 = w.s0;
    e.s = u.s;
    e.hk = head;
    e.t0 = u.t0;
    e.n = u.n;
    e.first = u.first;
    e.before = u.p0 - u.first;
    e.len = u.len;
    e.begins = i0 == 0;
    e.whole = i0 == 0 && i1 == cost;
    e.more = i1 == cost ? 0 : (int)div_pos(pos - i0 + cost - 1, per) - run;
    return e;
}

// The first segment of a run that begins `off` places behind a sequence's first head's
// first block; head_cost: the places of one head's blocks.
RA_HD TreeSegment tree_first_segment(const PagedSeqs &q, const TreeSeq &t, long long head_cost, int head0, long long off,
                                     long long pos, long long end, long long per, int run, int pad = 1) {
    const int head = (int)div_pos(off, head_cost);
    int i0 = (int)(off - head * head_cost), b = 0;
    for (int c; b + 1 < t.blocks && i0 >= (c = tree_block_cost(q, t, b, pad)); ++b) i0 -= c;
    return tree_segment(q, t, head0 + head, b, i0, pos, end, per, run, pad);
}
// The one after segment e, of the list of heads [head0, head0 + heads); t: e's sequence, then its own.
RA_HD TreeSegment tree_next_segment(const PagedSeqs &q, TreeSeq &t, const TreeSegment &e, int head0, int heads, long long pos,
                                    long long end, long long per, int run, int pad = 1) {
    int head = e.hk, b = e.first / q.unit_tokens + 1;
    if (b == t.blocks) {
        b = 0;
        if (++head == head0 + heads) {
            head = head0;
            do t = tree_seq(q, t.s + 1);
            while (t.blocks == 0);
        }
    }
    return tree_segment(q, t, head, b, 0, pos, end, per, run, pad);
}

}  // namespace ra
