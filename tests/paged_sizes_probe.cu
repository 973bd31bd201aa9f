// Test helper, not part of the library: the paged attention's sums over the
// sequences of a call at its largest sizes, on the host.
#include "paged_launch.h"

extern "C" {

// n sequences, the i-th with chunks[i % kinds] chunks: out gets the sequences
// counted that have any, and their chunks.
void ra_test_paged_tally(int64_t n, const int *chunks, int kinds, int64_t *out) {
    uint64_t sum = 0;
    for (int64_t i = 0; i < n; ++i) sum += ra::paged_tally(chunks[i % kinds]);
    out[0] = ra::paged_tally_seqs(sum);
    out[1] = ra::paged_tally_chunks(sum);
}

// The few-row form's grid; overflowing sums end the process where the compiler
// was asked for that.
int ra_test_paged_ctas(int64_t pairs, int64_t keys, int64_t n_seqs) { return ra::paged_tokens_ctas(pairs, keys, n_seqs); }

}  // extern "C"
