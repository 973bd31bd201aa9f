// Test helper, not part of the library: the same call from several host threads
// at once, `rounds` times each, with no lock between the calls.
#include <atomic>
#include <cstdint>
#include <thread>
#include <vector>

#include "ra.h"

namespace {

// failed[i]: how many of thread i's calls returned an error
template <class Call>
void at_once(int threads, int rounds, int *failed, Call call) {
    std::atomic<int> waiting{threads};
    std::vector<std::thread> pool;
    for (int i = 0; i < threads; ++i)
        pool.emplace_back([&, i] {
            --waiting;
            while (waiting > 0) std::this_thread::yield();
            int bad = 0;
            for (int r = 0; r < rounds; ++r) bad += call(i) != RA_OK;
            failed[i] = bad;
        });
    for (auto &t : pool) t.join();
}

}  // namespace

extern "C" {

// Thread i: its window, outputs, workspace and stream; d, q, k, v and the sizes are shared.
void ra_test_window_threads(decltype(&ra_window_attn_fwd) fn, int threads, int rounds, int *failed, const void *q,
                            const void *k, const void *v, int64_t L, int64_t H, int64_t H_kv, int d,
                            const int64_t *window, void *const *o, float *const *lse, void *const *ws,
                            void *const *stream) {
    at_once(threads, rounds, failed, [&](int i) {
        return fn(q, k, v, o[i], lse[i], nullptr, 0, 1, L, H, H_kv, d, window[i], 0, 0.f, RA_FLAG_O_BF16, ws[i],
                  RA_WORKSPACE_MIN_BYTES, stream[i]);
    });
}

// Thread i: its max_len, outputs, workspace and stream; gapless pages, n_seqs sequences of max_new tokens each.
void ra_test_paged_threads(decltype(&ra_paged_attn_fwd) fn, int threads, int rounds, int *failed, const void *q,
                           const void *k, const void *v, const int32_t *table, const int32_t *lens, const int32_t *cu,
                           int64_t n_seqs, int64_t max_new, int64_t H, int64_t H_kv, int d, int64_t n_pages,
                           int64_t page, int64_t max_pages, const int64_t *max_len, void *const *o, float *const *lse,
                           void *const *ws, size_t ws_bytes, void *const *stream) {
    at_once(threads, rounds, failed, [&](int i) {
        return fn(q, k, v, table, lens, cu, o[i], lse[i], n_seqs * max_new, n_seqs, H, H_kv, d, n_pages, page,
                  page * H_kv * d, max_pages, H * d, max_new, max_len[i], 0, 0, 0.f, RA_FLAG_O_BF16, ws[i], ws_bytes,
                  stream[i]);
    });
}

}  // extern "C"
