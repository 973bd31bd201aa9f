// ra_tensor_map.h -- the driver's tensor-map encoder, looked up once, and the
// maps of the attention kernels' tiles.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "ra_internal.h"

namespace ra {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn get_encode_fn() {
    static EncodeTiledFn fn = nullptr;
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    }
    return fn;
}

// The 4-D view `tv` of a [..., cols] bf16 (or fp32) tensor, in boxes of 128
// bytes of columns by 128 rows with the 128-byte swizzle the operand
// descriptors (and the O staging) expect.
inline bool tile_map(CUtensorMap *map, const void *base, const TileView &tv, int64_t cols, bool f32 = false) {
    EncodeTiledFn enc = get_encode_fn();
    if (!enc) return false;
    const cuuint64_t esz = f32 ? 4 : 2;
    cuuint64_t dims[4] = {(cuuint64_t)cols, (cuuint64_t)tv.n[0], (cuuint64_t)tv.n[1], (cuuint64_t)tv.n[2]};
    cuuint64_t strides[3] = {(cuuint64_t)tv.st[0] * esz, (cuuint64_t)tv.st[1] * esz, (cuuint64_t)tv.st[2] * esz};
    cuuint32_t box[4] = {(cuuint32_t)(128 / esz), tv.row_dim == 0 ? 128u : 1u, tv.row_dim == 1 ? 128u : 1u, 1u};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
               const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace ra
