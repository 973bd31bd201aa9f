// Test helper, not part of the library: runs the windowed attention's own
// tile walk, row keys and sink units (ra_window.cuh) on the host and counts,
// for every (query, key) pair, how often the kernels let it through.
#include "ra_window.cuh"

extern "C" {

// cnt[p * S + t]: how often the walk of a `rows`-row unit, masked per row,
// gives key t to query p (forward: 256 rows, dQ pass: 128).
void ra_test_window_rows(int S, int window, int sinks, const int *cu, int n_seqs, int rows, int *cnt) {
    for (int row0 = 0; row0 < S; row0 += rows) {
        const int row_end = row0 + rows < S ? row0 + rows : S;
        ra::RangeWalk w = ra::window_unit_walk(cu, n_seqs, S, row0, row_end, window, sinks);
        for (w.start_step(); w.valid(); w.next())
            for (int p = row0; p < row_end; ++p) {
                const ra::RowKeys k = ra::window_row(cu, n_seqs, S, p, window, sinks);
                for (int t = w.tile * 128; t < w.tile * 128 + 128 && t < S; ++t)
                    if ((t >= k.lo && t < k.hi) || (t >= k.slo && t < k.shi)) ++cnt[(size_t)p * S + t];
            }
    }
}

// cnt[u * 256 + r]: how often the forward's blocks have row r of unit u.
// Returns the number of blocks of a launch, or -1 if one leaves the units.
int ra_test_window_units(int units, int sms, int *cnt) {
    const int whole = (int)ra::window_whole_units(units, sms), blocks = 2 * units - whole;
    for (int i = 0; i < blocks; ++i) {
        const ra::WindowRows w = ra::window_rows(i, whole);
        if (w.unit < 0 || w.unit >= units) return -1;
        for (int r = 0; r < w.rows(); ++r) ++cnt[w.unit * 256 + w.first(0) + r];
    }
    return blocks;
}

// The same for the dK / dV pass: each key against the queries of its window,
// in 128-query tiles of its block's walk, and each sink against the units past
// its window; a unit's partial counts only if the key's sum reads it.
// Returns 1 if a unit number leaves [0, sink_units).
int ra_test_window_cols(int S, int window, int sinks, const int *cu, int n_seqs, int slot_bytes, int *cnt) {
    const int chunk = ra::sink_chunk(window, S, cu ? n_seqs : 0, slot_bytes);
    const int64_t units = ra::sink_units(S, cu ? n_seqs : 0, chunk);
    for (int c0 = 0; c0 < S; c0 += 128) {
        const int c_end = c0 + 128 < S ? c0 + 128 : S;
        int start, end;
        ra::seq_of(cu, n_seqs, S, c_end - 1, start, end);
        const int last = ra::window_col_end(c_end - 1, end, window);
        for (int t = c0; t < c_end; ++t) {
            const int s = ra::seq_of(cu, n_seqs, S, t, start, end);
            const int hi = ra::window_col_end(t, end, window);
            for (int p = c0 / 128 * 128; p < (last + 127) / 128 * 128; ++p)
                if (p >= t && p < hi) ++cnt[(size_t)p * S + t];
            if (t - start >= sinks || t + window >= end) continue;
            for (int u = s + (t + window) / chunk; u < s + (end - 1) / chunk + 1; ++u) {
                if (u < 0 || u >= units) return 1;
                const ra::SinkUnit k = ra::sink_unit(cu, n_seqs, S, chunk, u);
                if (k.start != start || k.end != end) return 2;
                // the unit's block holding t must have run: its first key has a query in the chunk
                const int b0 = start + (t - start) / 128 * 128;
                if ((k.lo > b0 + window ? k.lo : b0 + window) >= k.hi) return 3;
                for (int p = k.lo > t + window ? k.lo : t + window; p < k.hi; ++p) ++cnt[(size_t)p * S + t];
            }
        }
    }
    return 0;
}
}
