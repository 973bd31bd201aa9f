// attn_paged_tree.cu -- the launches of tree attention: the few-row form
// (attn_paged_tokens.cuh) and the tensor-core form (attn_tree.cuh).  The entry
// point, its checks and its plan are in attn_paged.cu; the kernels in parts in
// attn_paged_tree_long.cu, to be compiled beside these.
#include "attn_paged_tokens.cuh"
#include "attn_tree.cuh"

namespace ra {

ra_status launch_tree_tokens(const TokensLaunch &t, const TokensArgs &a, cudaStream_t stream) {
    return launch_tokens<true>(t, a, stream);
}

ra_status launch_tree(const TreeLaunch &t, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                      cudaStream_t stream) {
    TreeArgs a{};
    a.seqs = t.seqs;
    a.tile_tokens = t.tile_tokens;
    a.page_box = t.page_box;
    a.two = t.two;
    a.min_run = kTreeMinRun;
    a.streams = t.streams;
    a.heads = t.seqs.Hkv / t.streams;
    a.scale_log2 = t.scale_log2;
    a.status = t.status;
    a.o = t.o;
    a.lse = t.lse;
    a.o_bf16 = t.o_bf16;
    a.part_o = static_cast<float4 *>(t.part_o);
    a.part_ml = static_cast<float4 *>(t.part_ml);
    a.cuts = static_cast<TreeCut *>(t.cuts);
    // few units to a stream are cut into many pieces
    const bool many = t.units * 6 < t.ctas;
    auto go = [&](auto kern, auto join, int smem) -> ra_status {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return set_error(RA_ERR_CUDA, "cudaFuncSetAttribute(MaxDynamicSharedMemorySize) failed");
        const ra_status st = launched(launch_dependent(kern, (unsigned)t.ctas, 384, smem, stream, q, k, v, a));
        if (st != RA_OK || t.ctas == t.streams) return st;       // one run to a stream cuts no unit
        return launched(launch_dependent(join, (unsigned)(many ? kTreeCtas : 3 * kTreeCtas), 256, 0, stream, a, t.ctas));
    };
    const TreeKernel parts = t.in_parts ? tree_kernel_in_parts(t.d, t.two) : nullptr;
    if (t.d == 128)
        return go(parts ? parts : t.two ? paged_tree_kernel<128, true, false> : paged_tree_kernel<128, false, false>,
                  many ? paged_tree_join_kernel<128, 10> : paged_tree_join_kernel<128, 4>, (int)TreeSmem<128, true>::kBytes);
    return go(parts ? parts : t.two ? paged_tree_kernel<64, true, false> : paged_tree_kernel<64, false, false>,
              many ? paged_tree_join_kernel<64, 10> : paged_tree_join_kernel<64, 4>, (int)TreeSmem<64, true>::kBytes);
}

}  // namespace ra
