// Test helper, not part of the library: the key tiles of tree attention's units, and which calls work
// on them in parts (paged_launch.h), on the host.
#include "paged_launch.h"
#include "ra_tree.cuh"

// The most tiles of a unit of one sequence of `len` tokens, n of them new.
extern "C" int ra_test_tree_tiles(int len, int n, int max_pages, int page, int unit_tokens, int max_new, int window, int sinks) {
    const int cu[2] = {0, n};
    int parents = 0;
    ra::PagedSeqs q{};
    q.seq_lens = &len;
    q.cu_q = cu;
    q.parents = &parents;
    q.n_seqs = 1;
    q.T = n;
    q.max_pages = max_pages;
    q.page = page;
    q.H = q.Hkv = q.group = 1;
    q.unit_tokens = unit_tokens;
    q.max_new = max_new < n ? max_new : n;
    q.window = window;
    q.sinks = sinks;
    const ra::TreeSeq t = ra::tree_seq(q, 0);
    int most = 0;
    for (int b = 0; b < t.blocks; ++b) {
        const int cost = ra::tree_block_cost(q, t, b);
        most = cost > most ? cost : most;
    }
    return most;
}

extern "C" int ra_test_tree_in_parts(long long capacity, long long max_new, long long window, long long sinks) {
    return ra::tree_in_parts(capacity, max_new, window, sinks) ? ra::kTreePart : -ra::kTreePart;
}
