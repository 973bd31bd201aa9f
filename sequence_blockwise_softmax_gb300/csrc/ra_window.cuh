// ra_window.cuh -- which keys a row of windowed attention sees, and the key
// tiles a block of rows visits; the paged form's units and splits.
//
// Plain integer arithmetic callable from host and device, as in
// ra_positions.cuh, so that a CPU test can run what the kernels run
// (tests/window_probe.cu).
//
// A query at position p of a sequence that starts at `start` sees the keys t
// of its sequence with t <= p and (t > p - window or t < start + sinks): an
// interval that ends at the query, and the sinks it has left behind.
#pragma once
#include <cstdint>

#include "ra_positions.cuh"

namespace ra {

// The tokens that belong to sequences: up to the last boundary, or all L.  Rows
// behind them are neither read into a result nor written.
RA_HD int packed_tokens(const int *cu, int n_seqs, int L) { return cu ? (int)clamp64(cu[n_seqs], 0, L) : L; }

// Boundary i of the packed sequences over S tokens, i in [0, n_seqs + 1] (what
// lies past the last boundary, if anything, is one more sequence).  Every read
// stays inside the n_seqs + 1 boundaries and every value inside [0, S],
// whatever they hold.
RA_HD int seq_bound(const int *cu, int n_seqs, int S, int i) {
    return i > n_seqs ? S : (int)clamp64(cu[i], 0, S);
}

// The number of the sequence holding position p, and its bounds; without
// packing (cu null) number 0, [0, S).
RA_HD int seq_of(const int *cu, int n_seqs, int S, int p, int &start, int &end) {
    start = 0;
    end = S;
    if (!cu) return 0;
    int lo = 0, hi = n_seqs + 1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seq_bound(cu, n_seqs, S, mid) <= p) lo = mid;
        else hi = mid;
    }
    start = seq_bound(cu, n_seqs, S, lo);
    end = seq_bound(cu, n_seqs, S, lo + 1);
    if (start > p) start = p;
    if (end < p + 1) end = p + 1;
    return lo;
}

// The keys of one row: [lo, hi) and, when the window has left the sinks
// behind, [slo, shi) with shi < lo; otherwise slo = shi = 0 and [lo, hi) holds
// both.  hi <= lo for a row that sees nothing (a negative position).
struct RowKeys {
    int lo, hi, slo, shi;
};

// window <= 0 means no window.  Everything lies in [0, 2^30], so no sum here
// leaves 32 bits.
RA_HD RowKeys window_row_keys(int start, int p, int window, int sinks) {
    RowKeys r;
    r.hi = p + 1;
    r.lo = window > 0 && p - window + 1 > start ? p - window + 1 : start;
    r.slo = r.shi = 0;
    const int s_end = start + sinks < p + 1 ? start + sinks : p + 1;
    if (r.lo > start && s_end > start) {
        if (s_end >= r.lo) {
            r.lo = start;
        } else {
            r.slo = start;
            r.shi = s_end;
        }
    }
    return r;
}

// The key tiles (128 keys) a block of rows visits, in order: n_sink tiles from
// s0 on, then tiles from m0 on; tile number i of `end` in all, from `i` on.
// The rows' positions increase and `first` is the first row's keys, so that
// the main tiles run from first.lo to the last row's position: a later row's
// window starts no earlier, a later sequence's sinks lie after first.lo, and
// sinks left behind by a row of the first sequence are first's (or lie after
// first.lo = start).
struct RangeWalk {
    int i, end, n_sink, s0, m0;
    int tile, j;

    RA_HD_STEP void seek() { tile = i < n_sink ? s0 + i : m0 + (i - n_sink); }
    RA_HD_STEP void start_step() { seek(); }
    RA_HD_STEP bool valid() const { return i < end; }
    RA_HD_STEP void next() {
        ++i;
        seek();
    }
};

RA_HD RangeWalk range_walk(const RowKeys &first, int last_hi) {
    RangeWalk w;
    w.j = 0;
    w.i = 0;
    w.m0 = first.lo / 128;
    const int m1 = (last_hi + 127) / 128;
    w.s0 = first.slo / 128;
    int s1 = (first.shi + 127) / 128;
    if (s1 > w.m0) s1 = w.m0;
    w.n_sink = first.shi > first.slo && s1 > w.s0 ? s1 - w.s0 : 0;
    w.end = w.n_sink + (m1 > w.m0 ? m1 - w.m0 : 0);
    w.tile = 0;
    return w;
}

// The walk of a unit of windowed rows [row0, row_end) of one batch element of
// S tokens (packed sequences: cu, n_seqs).
RA_HD RowKeys window_row(const int *cu, int n_seqs, int S, int p, int window, int sinks) {
    int start, end;
    seq_of(cu, n_seqs, S, p, start, end);
    return window_row_keys(start, p, window, sinks);
}

// Block number `block` of the forward: whole units of 256 rows, then the rest
// in halves of 128 rows.
struct WindowRows {
    int unit, half;     // half < 0: the whole unit
    RA_HD int first(int row0) const { return half > 0 ? row0 + 128 : row0; }    // row0: the unit's
    RA_HD int rows() const { return half < 0 ? 256 : 128; }
};
RA_HD WindowRows window_rows(int block, int whole) {
    const int rest = block - whole;
    return rest < 0 ? WindowRows{block, -1} : WindowRows{whole + rest / 2, rest & 1};
}
// The whole units of a call's `units` on `sms` SMs: none where an SM for each
// half is there.  A half takes about two thirds of a unit's time: 1024 tokens, 8
// heads, window 600: 15.7 us against 18.6 at d = 128, 12.5 against 16.1 at d =
// 64; 2048 tokens, window 1024: 20.0 against 22.9.  (Halves for the last wave of
// a longer call cost more than they even out, since its units are the lightest:
// 3000 tokens, 16 heads, window 1024: 33.9 against 29.2; 8192: 78 against 80.)
RA_HD int64_t window_whole_units(int64_t units, int sms) { return 2 * units <= sms ? 0 : units; }

RA_HD RangeWalk window_unit_walk(const int *cu, int n_seqs, int S, int row0, int row_end, int window, int sinks) {
    return range_walk(window_row(cu, n_seqs, S, row0, window, sinks), row_end);
}

// The key tiles that some row of a block of consecutive rows sees (its first
// row's keys, one past its last row's position): tiles [m0, m1) and, of the
// sinks left behind, [s0, s1).
struct SeenTiles {
    int m0, m1, s0, s1;
    RA_HD bool has(int tile) const { return (tile >= m0 && tile < m1) || (tile >= s0 && tile < s1); }
};
RA_HD SeenTiles seen_tiles(const RowKeys &first, int last_hi) {
    SeenTiles t;
    t.m0 = first.lo / 128;
    t.m1 = (last_hi + 127) / 128;
    t.s0 = first.slo / 128;
    t.s1 = first.shi > first.slo ? (first.shi + 127) / 128 : t.s0;
    return t;
}

// The queries that meet a key at position t inside the window: rows [t, hi),
// hi = t + window but not past the end of t's sequence.
RA_HD int window_col_end(int t, int end, int window) {
    return window > 0 && end - t > window ? t + window : end;
}

// The far part of a sink's gradient: the queries past its window.  They are
// cut at multiples of `chunk` rows and each (sequence, chunk) is a unit of
// its own, so that the few keys every query sees do not become one long block.
// Unit u belongs to the last sequence s whose first unit, start / chunk + s,
// is not past u, and is chunk u - s of the rows; the chunks of a sequence
// [start, end) are start / chunk .. (end - 1) / chunk, one more than
// the next sequence's start is on at most, which the "+ s" has room for.
// A chunk is about as long as a key block's own queries (the window), so that
// the two kinds of block take alike, from 512 rows (shorter ones cost more CTAs
// than they even out: 3000 tokens, window 100, 36 us with 256 against 32) to
// 2048; longer where the partial gradients (slot_bytes for each unit and each
// sequence) would pass 32 MiB.  Where the two slots of each sequence pass that by
// themselves no length keeps inside it, and one chunk holds all S rows: the far
// queries of a sequence are then one block, in (2 n_seqs + 3) slots at most.
RA_HD int sink_chunk(int64_t window, int64_t S, int64_t n_seqs, int64_t slot_bytes) {
    int64_t c = window <= 512 ? 512 : window >= 2048 ? 2048 : (window + 127) / 128 * 128;
    while (c < S && (S / c + 2 * n_seqs + 2) > ((int64_t)32 << 20) / (slot_bytes > 0 ? slot_bytes : 1)) c *= 2;
    return (int)c;
}

struct SinkUnit {
    int start, end;     // the sequence's tokens
    int lo, hi;         // the chunk's query rows inside it; lo >= hi: no such unit
};

RA_HD int64_t sink_units(int64_t S, int n_seqs, int chunk) { return S / chunk + n_seqs + 1; }

// The number of the first unit of sequence s, which starts at `start`.
RA_HD int sink_first_unit(int start, int s, int chunk) { return start / chunk + s; }

RA_HD SinkUnit sink_unit(const int *cu, int n_seqs, int S, int chunk, int u) {
    SinkUnit k;
    int s = 0;
    k.start = 0;
    k.end = S;
    if (cu) {
        int hi = n_seqs + 1;
        while (hi - s > 1) {
            const int mid = (s + hi) >> 1;
            if (sink_first_unit(seq_bound(cu, n_seqs, S, mid), mid, chunk) <= u) s = mid;
            else hi = mid;
        }
        k.start = seq_bound(cu, n_seqs, S, s);
        k.end = seq_bound(cu, n_seqs, S, s + 1);
    }
    const int64_t at = (int64_t)(u - s) * chunk;   // unit start / chunk + s + i is chunk start / chunk + i
    k.lo = (int)clamp64(at, k.start, k.end);
    k.hi = (int)clamp64(at + chunk, k.start, k.end);
    return k;
}

}  // namespace ra
