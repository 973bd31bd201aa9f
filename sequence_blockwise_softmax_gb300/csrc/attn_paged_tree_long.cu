// attn_paged_tree_long.cu -- tree attention's tensor-core kernels for long units, which are
// worked on in parts (attn_tree.cuh).
#include "attn_tree.cuh"

namespace ra {

TreeKernel tree_kernel_in_parts(int d, bool two) {
    if (d == 128) return two ? paged_tree_kernel<128, true, true> : paged_tree_kernel<128, false, true>;
    return two ? paged_tree_kernel<64, true, true> : paged_tree_kernel<64, false, true>;
}

}  // namespace ra
