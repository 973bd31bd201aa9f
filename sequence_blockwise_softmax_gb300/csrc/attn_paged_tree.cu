// attn_paged_tree.cu -- the tree forms of paged attention's kernels: the few-row
// form (attn_paged_tokens.cuh) and the tensor-core form (attn_fwd_kernel.cuh,
// KEYS_TREE).  The entry point is in attn_paged.cu.
#include "attn_fwd_kernel.cuh"
#include "attn_paged_tokens.cuh"

namespace ra {

ra_status launch_tree_tokens(const TokensLaunch &t, const TokensArgs &a, cudaStream_t stream) {
    return launch_tokens<true>(t, a, stream);
}

AttnKernel tree_chunk_kernel(int d, bool f32, int *smem) {
    *smem = (int)(d == 128 ? AttnSmem<128>::kBytesTree : AttnSmem<64>::kBytesTree);
    static_assert(AttnSmem<128>::kBytesTree <= 232448, "what a CTA may have");
    if (d == 128) return f32 ? attn_fwd_kernel<128, true, false, KEYS_TREE> : attn_fwd_kernel<128, false, false, KEYS_TREE>;
    return f32 ? attn_fwd_kernel<64, true, false, KEYS_TREE> : attn_fwd_kernel<64, false, false, KEYS_TREE>;
}

}  // namespace ra
