// attn_paged_tokens.cu -- the few-row form's launch (attn_paged_tokens.cuh).
#include <atomic>

#include "attn_paged_tokens.cuh"

namespace ra {

ra_status launch_paged_tokens(const TokensLaunch &t, cudaStream_t stream) {
    TokensArgs a{};
    a.seqs = t.seqs;
    a.q = static_cast<const uint16_t *>(t.q);
    a.k = static_cast<const uint16_t *>(t.k);
    a.v = static_cast<const uint16_t *>(t.v);
    a.q_stride = t.q_stride;
    a.page_stride = t.page_stride;
    a.o = t.o;
    a.lse = t.lse;
    a.o_bf16 = t.o_bf16;
    a.whole_pairs = t.whole_pairs;
    a.row_blocks = t.row_blocks;
    a.scale_log2 = t.scale_log2;
    a.status = t.status;
    static std::atomic<unsigned long long> calls{0};
    a.call = call_tag(calls.fetch_add(1, std::memory_order_relaxed));
    a.counters = t.counters;
    a.part_o = t.part_o;
    a.part_ml = t.part_ml;
    return t.seqs.parents ? launch_tree_tokens(t, a, stream) : launch_tokens<false>(t, a, stream);
}

}  // namespace ra
