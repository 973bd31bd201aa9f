// attn_sm103.cu -- launches of the ring form of the forward kernel
// (attn_fwd_kernel.cuh): its tensor maps, arguments and variants.
#include <cmath>
#include <cstdio>

#include "attn_fwd_kernel.cuh"
#include "ra_tensor_map.h"

namespace ra {

// The 4-D view tile_view describes, for a [..., heads * d] tensor of the launch.
static bool make_map(CUtensorMap *map, const void *base, const AttnLaunch &a, int64_t heads, int d,
                     bool f32 = false) {
    return tile_map(map, base, tile_view(a.seq_order, a.layout, a.S, a.B, a.N, a.ring ? a.N : 1, heads * d),
                    heads * d, f32);
}

template <int D, bool F32, bool SKIP>
static ra_status launch_t(const AttnLaunch &a, const AttnArgs &args, int64_t grid, cudaStream_t stream,
                          const char **err) {
    CUtensorMap mq, mk, mv, mo;
    const int64_t Hkv = a.H_kv > 0 ? a.H_kv : a.H;
    if (!make_map(&mq, a.q, a, a.H, D) || !make_map(&mk, a.k, a, Hkv, D) || !make_map(&mv, a.v, a, Hkv, D) ||
        !make_map(&mo, a.o, a, a.H, D, F32)) {
        *err = "cuTensorMapEncodeTiled failed for the q/k/v/o tensor maps";
        return RA_ERR_CUDA;
    }
    auto kern = attn_fwd_kernel<D, F32, SKIP>;
    const int smem = (int)(SKIP ? AttnSmem<D>::kBytesSkip : AttnSmem<D>::kBytes);
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
        *err = "cudaFuncSetAttribute(MaxDynamicSharedMemorySize) failed";
        return RA_ERR_CUDA;
    }
    kern<<<(unsigned)grid, 384, smem, stream>>>(mq, mk, mv, mo, args);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        *err = cudaGetErrorString(e);
        return RA_ERR_CUDA;
    }
    return RA_OK;
}

ra_status launch_attention(const AttnLaunch &a, cudaStream_t stream, const char **err) {
    AttnArgs args;
    args.o = a.o;
    args.lse = a.lse;
    args.status = a.status;
    args.B = (int)a.B;
    args.S = (int)a.S;
    args.H = (int)a.H;
    args.N = a.N;
    args.layout = a.layout;
    args.causal = a.causal ? 1 : 0;
    const float scale = a.scale > 0.f ? a.scale : 1.0f / std::sqrt((float)a.d);
    args.scale_log2 = scale * 1.4426950408889634f;
    args.num_q_ranks = a.ring ? a.N : 1;
    args.q_rank_fixed = a.ring ? -1 : a.q_rank;
    args.kv_rank_fixed = a.ring ? -1 : a.kv_rank;
    args.num_steps = (a.ring && a.ring_step < 0) ? a.N : 1;
    args.step_base = a.ring_step < 0 ? 0 : a.ring_step;
    args.n_units_seq = (int)((a.S + 255) / 256);
    args.inject_stall = a.inject_stall ? 1 : 0;
    args.kv_group = (int)(a.H / (a.H_kv > 0 ? a.H_kv : a.H));
    args.cu_seqlens = a.cu_seqlens;
    args.n_seqs = a.n_seqs;
    // keys + values one query head sweeps, shared by the heads of a GQA group;
    // a chunk holds about 48 MB of them by default (L2 holds 129 MB)
    args.bh_chunk = chunk_pairs(2 * (a.ring ? a.N : 1) * a.S * a.d * 2 / args.kv_group, a.B * a.H);
    args.seq_order = a.seq_order ? 1 : 0;
    const int64_t grid = (int64_t)args.num_q_ranks * args.n_units_seq * a.B * a.H;
    if (grid == 0) return RA_OK;
    if (grid > 0x7fffffffLL) {
        *err = "too many query tiles for one launch";
        return RA_ERR_UNSUPPORTED;
    }
    // Packed sequences in the striped layout take the tile-skipping variant
    // (d = 128): there a unit's 256 rows span N x 256 positions, many short
    // sequences, and each Q tile sees few of the tiles the unit visits.
    // Elsewhere skipping removes little work and measured slower (zigzag
    // packed sequences too).
    const bool skip = a.d == 128 && a.cu_seqlens != nullptr && a.layout == RA_STRIPED;
    if (skip)
        return a.out_f32 ? launch_t<128, true, true>(a, args, grid, stream, err)
                         : launch_t<128, false, true>(a, args, grid, stream, err);
    if (a.d == 128)
        return a.out_f32 ? launch_t<128, true, false>(a, args, grid, stream, err)
                         : launch_t<128, false, false>(a, args, grid, stream, err);
    return a.out_f32 ? launch_t<64, true, false>(a, args, grid, stream, err)
                     : launch_t<64, false, false>(a, args, grid, stream, err);
}

}  // namespace ra
