// attn_bwd_sm103.cu -- launches of the ring form of the backward kernels
// (attn_bwd_kernels.cuh).
#include <cmath>

#include "attn_bwd_kernels.cuh"
#include "ra_tensor_map.h"

namespace ra {

// The 4-D view tile_view describes (shard stacks or token order).
static bool bwd_map(CUtensorMap *map, const void *base, const BwdLaunch &a, int64_t heads, int d) {
    return tile_map(map, base, tile_view(a.seq_order, a.layout, a.S, a.B, a.N, a.N, heads * d), heads * d);
}

template <int D>
static ra_status bwd_launch_t(const BwdLaunch &a, BwdArgs args, cudaStream_t stream, const char **err) {
    const int64_t Z = (int64_t)a.N * a.B;
    CUtensorMap mq, mk, mv, mdo;
    if (!bwd_map(&mq, a.q, a, a.H, D) || !bwd_map(&mk, a.k, a, a.H_kv, D) || !bwd_map(&mv, a.v, a, a.H_kv, D) ||
        !bwd_map(&mdo, a.dout, a, a.H, D)) {
        *err = "cuTensorMapEncodeTiled failed for the backward tensor maps";
        return RA_ERR_CUDA;
    }
    // D = rowsum(dO * O) (and, in token order, the stack-order LSE copy)
    {
        const int64_t rows = Z * a.S * a.H;
        int dev = 0, sms = 148;
        cudaGetDevice(&dev);
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        int64_t blocks = (rows + 31) / 32;   // 8 warps of 4 rows
        if (blocks > (int64_t)sms * 8) blocks = (int64_t)sms * 8;
        bwd_dot_kernel<D><<<(unsigned)blocks, 256, 0, stream>>>(static_cast<const uint16_t *>(a.dout), a.o,
                                                                 a.dvec, rows, (int)a.H, a.S, a.seq_order ? 1 : 0,
                                                                 a.layout, a.N, (int)a.B, a.lse, a.lse_stack);
    }
    auto kq = attn_bwd_dq_kernel<D>;
    auto kkv = attn_bwd_dkv_kernel<D>;
    if (cudaFuncSetAttribute(kq, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)BwdQSmem<D>::kBytes) !=
            cudaSuccess ||
        cudaFuncSetAttribute(kkv, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)BwdKVSmem<D>::kBytes) !=
            cudaSuccess) {
        *err = "cudaFuncSetAttribute(MaxDynamicSharedMemorySize) failed";
        return RA_ERR_CUDA;
    }
    const int64_t grid_kv = Z * a.H_kv * args.n_tiles_seq;
    const int64_t grid_q = Z * a.H * args.n_tiles_seq;
    if (grid_kv > 0x7fffffffLL || grid_q > 0x7fffffffLL) {
        *err = "too many tiles for one launch";
        return RA_ERR_UNSUPPORTED;
    }
    kkv<<<(unsigned)grid_kv, 384, BwdKVSmem<D>::kBytes, stream>>>(mq, mk, mv, mdo, args);
    kq<<<(unsigned)grid_q, 384, BwdQSmem<D>::kBytes, stream>>>(mq, mk, mv, mdo, args);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        *err = cudaGetErrorString(e);
        return RA_ERR_CUDA;
    }
    return RA_OK;
}

ra_status launch_attention_bwd(const BwdLaunch &a, cudaStream_t stream, const char **err) {
    BwdArgs args;
    args.lse = a.seq_order ? a.lse_stack : a.lse;
    args.dvec = a.dvec;
    args.dq = a.dq;
    args.dk = a.dk;
    args.dv = a.dv;
    args.status = a.status;
    args.cu_seqlens = a.cu_seqlens;
    args.n_seqs = a.n_seqs;
    args.B = (int)a.B;
    args.S = (int)a.S;
    args.H = (int)a.H;
    args.Hkv = (int)a.H_kv;
    args.N = a.N;
    args.layout = a.layout;
    args.causal = a.causal ? 1 : 0;
    args.scale = a.scale > 0.f ? a.scale : 1.0f / std::sqrt((float)a.d);
    args.scale_log2 = args.scale * 1.4426950408889634f;
    args.n_tiles_seq = (int)((a.S + 127) / 128);
    args.seq_order = a.seq_order ? 1 : 0;
    if ((int64_t)a.N * a.B * a.S * a.H == 0) return RA_OK;
    {
        // bytes a tile's sweep streams per (batch, head) pair: keys + values
        // per query head in the dQ pass (shared by a GQA group), queries + dO
        // of the whole group per key/value head in the dK/dV pass
        const int64_t group = a.H / a.H_kv;
        const int64_t per_head = 2 * (int64_t)a.N * a.S * a.d * 2;
        args.bh_chunk_q = chunk_pairs(per_head / group, a.B * a.H);
        args.bh_chunk_kv = chunk_pairs(per_head * group, a.B * a.H_kv);
    }
    return a.d == 128 ? bwd_launch_t<128>(a, args, stream, err) : bwd_launch_t<64>(a, args, stream, err);
}

}  // namespace ra
