// attn_window.cu -- causal sliding-window attention with sinks, forward and
// backward: the entry points, their checks and launches.  The kernels are the
// ring sweep's (attn_fwd_kernel.cuh, attn_bwd_kernels.cuh) with N = 1 and the
// keys of ra_window.cuh: a unit of 256 query rows visits the key tiles its
// window covers and the tile or two that hold its sequence's first tokens.
//
// Forward: bound by a unit's fixed 7 us (set-up, first loads, epilogue) beside
// about 1.3 us a tile, the tensor cores' own pace inside the loop: 128K tokens, 8
// heads, d = 128, window 1024: 592 us (980 TFLOP/s over the visible pairs), 8192
// tokens, 16 heads: 80 us, 67 at d = 64; window 4096 over 32K tokens, 8 heads: 376
// us (1370 TFLOP/s).
// Backward: 7 products for the 5 that the formulas need (both passes rebuild S
// and dP): 32K tokens, 8 heads, d = 128, window 2048, 128 sinks: 838 us (1180
// TFLOP/s executed); 8191 packed tokens, 16 / 4 heads, d = 64, window 500: 128 us,
// where the CTAs are short.  These are calls one after another on other inputs each
// time; on the same inputs again, part of them in L2, 569, 804 and 127 us.
#include <cmath>

#include "attn_bwd_kernels.cuh"
#include "attn_fwd_kernel.cuh"
#include "ra_launch.h"
#include "ra_tensor_map.h"
#include "window_few.h"

namespace ra {
namespace {

constexpr size_t kHeader = RA_WORKSPACE_MIN_BYTES;
constexpr int kSms = 152;     // GB300; only choices of a form depend on it
constexpr int kMostSeqs = 1 << 29;   // two of them and the sinks' units stay inside 32 bits
size_t round256(size_t x) { return (x + 255) & ~size_t(255); }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The few-key form runs where 16 rows meet few 16-key chunks.  Few-key against
// tensor-core form in us, four sinks:
//   Its warps sharing 16 rows, 512 tokens, 2 heads, d = 64: window 128: 4.1 / 7.6,
//   400: 6.0 / 8.0; d = 128, 300: 7.2 / 9.9; 8 heads, d = 64, 300: 6.6 / 8.2.  Else
//   512 tokens, 8 / 2 heads (one wave of CTAs), d = 64: window 16: 3.7 / 7.8,
//   128: 6.0 / 7.8, 200: 7.8 / 8.6, 300: 9.7 / 8.3; d = 128: 4.6 / 9.4,
//   7.8 / 9.2, 10.1 / 10.5, 12.7 / 10.0.
//   2000 tokens, 8 / 8 heads, d = 128: 6.0 / 10.7 and, where an SM holds one
//   CTA, not two, 14.8 / 10.5.
//   40000 tokens, 16 / 8 heads, d = 64: 80 / 167, 157 / 165, 257 / 185; d = 128:
//   window 16: 142 / 201, 64: 201 / 200, 128: 424 / 200.
bool few_keys(int64_t B, int64_t L, int64_t H, int d, int window, int sinks) {
    const int64_t row_chunks = ((int64_t)window + 30) / 16 + ((int64_t)sinks + 15) / 16;
    if (window_few_split(B, L, H, d, window, sinks)) return true;
    const size_t smem = window_few_smem(window_few_chunks((int)L, window, sinks, false), d, false), most = (size_t)227 << 10;
    const bool one_wave = B * H * ((L + 63) / 64) <= (2 * (smem + 1024) <= most + 1024 ? 2 * kSms : kSms);
    return row_chunks <= (one_wave ? 16 : d == 64 ? 11 : 5) && smem <= kWindowFewSmem;
}

struct Window {
    int64_t B, L, H, H_kv;
    int d, window, sinks;   // clipped to L
    float scale;
    const int *cu;
    int n_seqs;
};

// [B, L, heads, d] seen as the ring kernels' one-shard stack
TileView view(const Window &w, int64_t heads) { return tile_view(false, RA_CONTIGUOUS, w.L, w.B, 1, 1, heads * w.d); }

ra_status check(Window &w, int64_t window, int64_t sinks, const int *cu_seqlens, int n_seqs) {
    const ra_status st = check_attn_sizes(w.B, w.L, w.H, w.d, 1, RA_CONTIGUOUS, w.scale);
    if (st != RA_OK) return st;
    // positions plus a window or the sinks stay inside 32 bits
    if (w.L > ((int64_t)1 << 29)) return set_error(RA_ERR_UNSUPPORTED, "L beyond the supported range");
    if (w.H > 0 && (w.H_kv < 1 || w.H_kv > w.H || w.H % w.H_kv))
        return set_error(RA_ERR_SHAPE, "the key/value head count must divide the query head count");
    if (window < 1) return set_error(RA_ERR_INVALID_ARG, "window must be at least 1 (at least L: no window)");
    if (sinks < 0) return set_error(RA_ERR_INVALID_ARG, "sinks must not be negative");
    w.window = (int)(window < w.L ? window : w.L);
    w.sinks = (int)(sinks < w.L ? sinks : w.L);
    w.cu = cu_seqlens;
    w.n_seqs = 0;
    if (cu_seqlens) {
        if (w.B != 1) return set_error(RA_ERR_SHAPE, "packed sequences need B = 1");
        if (n_seqs < 1) return set_error(RA_ERR_SHAPE, "n_seqs must be at least 1");
        if (n_seqs > kMostSeqs) return set_error(RA_ERR_UNSUPPORTED, "n_seqs beyond the supported range (2^29)");
        if (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u)
            return set_error(RA_ERR_ALIGNMENT, "cu_seqlens must be 4-byte aligned");
        w.n_seqs = n_seqs;
    } else if (n_seqs != 0) {
        return set_error(RA_ERR_INVALID_ARG, "n_seqs without cu_seqlens");
    }
    if (w.B * w.H * ((w.L + 127) / 128) > 0x7fffffffLL)
        return set_error(RA_ERR_UNSUPPORTED, "too many query tiles for one launch");
    return RA_OK;
}

float softmax_scale(const Window &w) { return w.scale > 0.f ? w.scale : 1.0f / std::sqrt((float)w.d); }

template <int D, bool F32>
ra_status launch_fwd(const Window &w, const void *q, const void *k, const void *v, void *o, float *lse,
                     unsigned *status, cudaStream_t stream) {
    CUtensorMap mq, mk, mv, mo;
    if (!tile_map(&mq, q, view(w, w.H), w.H * D) || !tile_map(&mk, k, view(w, w.H_kv), w.H_kv * D) ||
        !tile_map(&mv, v, view(w, w.H_kv), w.H_kv * D) || !tile_map(&mo, o, view(w, w.H), w.H * D, F32))
        return set_error(RA_ERR_CUDA, "cuTensorMapEncodeTiled failed for the q/k/v/o tensor maps");
    AttnArgs a{};
    a.o = o;
    a.lse = lse;
    a.status = status;
    a.B = (int)w.B;
    a.S = (int)w.L;
    a.H = (int)w.H;
    a.N = 1;
    a.layout = RA_CONTIGUOUS;
    a.causal = 1;
    a.scale_log2 = softmax_scale(w) * 1.4426950408889634f;
    a.num_q_ranks = 1;
    a.q_rank_fixed = -1;
    a.kv_rank_fixed = -1;
    a.num_steps = 1;
    a.n_units_seq = (int)((w.L + 255) / 256);
    a.kv_group = (int)(w.H / w.H_kv);
    a.cu_seqlens = w.cu;
    a.n_seqs = w.n_seqs;
    a.bh_chunk = chunk_pairs(2 * w.L * D * 2 / a.kv_group, w.B * w.H);
    a.window = w.window;
    a.sinks = w.sinks;
    auto kern = attn_fwd_kernel<D, F32, false, KEYS_WINDOW>;
    const int smem = (int)AttnSmem<D>::kBytes;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return set_error(RA_ERR_CUDA, "cudaFuncSetAttribute(MaxDynamicSharedMemorySize) failed");
    const int64_t units = w.B * w.H * a.n_units_seq;
    a.whole_units = (int)window_whole_units(units, kSms);
    return launched(launch_dependent(kern, (unsigned)(2 * units - a.whole_units), 384, smem, stream, mq, mk, mv, mo, a));
}

// Workspace of the backward: the status word, D, the sinks' partial gradients.
struct BwdSpace {
    size_t dvec, part, total;
    int64_t units;
    int chunk;          // queries of a unit
};
BwdSpace bwd_space(int64_t B, int64_t L, int64_t H, int64_t H_kv, int d, int64_t window, int64_t sinks, int n_seqs) {
    BwdSpace s;
    if (sinks > L) sinks = L;
    // no query lies past a window of L tokens: no far part
    // (a slot past 2^46 bytes is refused below)
    const double slot = 8.0 * (double)B * (double)H_kv * (double)sinks * d;
    s.chunk = sink_chunk(window, L, n_seqs, slot < 0x1p46 ? (int64_t)slot : (int64_t)1 << 46);
    s.units = sinks > 0 && window < L ? sink_units(L, n_seqs, s.chunk) : 0;
    s.dvec = kHeader;
    const size_t slots = s.units > 0 ? s.units + (size_t)n_seqs + 1 : 0;
    // (sizes that no GPU holds would leave 64 bits)
    const unsigned __int128 rows = (unsigned __int128)B * L * H * 4,
                            part = (unsigned __int128)2 * B * H_kv * slots * sinks * d * 4;
    if (rows + part > ((unsigned __int128)1 << 46)) {
        s.part = s.total = 0;
        return s;
    }
    s.part = s.dvec + round256((size_t)rows);
    s.total = s.part + round256((size_t)part);
    return s;
}

template <int D>
ra_status launch_bwd(const Window &w, const void *q, const void *k, const void *v, const void *o, bool o_bf16,
                     const void *dout, const float *lse, void *dq, void *dk, void *dv, bool grad_bf16,
                     uint8_t *workspace, const BwdSpace &space, cudaStream_t stream) {
    CUtensorMap mq, mk, mv, mdo;
    if (!tile_map(&mq, q, view(w, w.H), w.H * D) || !tile_map(&mk, k, view(w, w.H_kv), w.H_kv * D) ||
        !tile_map(&mv, v, view(w, w.H_kv), w.H_kv * D) || !tile_map(&mdo, dout, view(w, w.H), w.H * D))
        return set_error(RA_ERR_CUDA, "cuTensorMapEncodeTiled failed for the backward tensor maps");
    BwdArgs a{};
    a.lse = lse;
    a.dvec = reinterpret_cast<float *>(workspace + space.dvec);
    a.dq = static_cast<float *>(dq);
    a.dk = static_cast<float *>(dk);
    a.dv = static_cast<float *>(dv);
    a.status = reinterpret_cast<unsigned *>(workspace);
    a.cu_seqlens = w.cu;
    a.n_seqs = w.n_seqs;
    a.B = (int)w.B;
    a.S = (int)w.L;
    a.H = (int)w.H;
    a.Hkv = (int)w.H_kv;
    a.N = 1;
    a.layout = RA_CONTIGUOUS;
    a.causal = 1;
    a.scale = softmax_scale(w);
    a.scale_log2 = a.scale * 1.4426950408889634f;
    a.n_tiles_seq = (int)((w.L + 127) / 128);
    const int64_t group = w.H / w.H_kv, per_head = 2 * w.L * D * 2;
    a.bh_chunk_q = chunk_pairs(per_head / group, w.B * w.H);
    a.bh_chunk_kv = chunk_pairs(per_head * group, w.B * w.H_kv);
    a.window = w.window;
    a.sinks = w.sinks;
    a.grad_bf16 = grad_bf16 ? 1 : 0;
    a.sink_units = (int)space.units;
    a.sink_part = reinterpret_cast<float *>(workspace + space.part);
    a.sink_chunk = space.chunk;
    const int64_t n_far = w.B * w.H_kv * ((w.sinks + 127) / 128) * space.units;
    const int64_t n_kv = w.B * w.H_kv * a.n_tiles_seq, n_q = w.B * w.H * a.n_tiles_seq;
    const int64_t joins = space.units > 0 ? w.B * w.H_kv * (w.n_seqs + 1) * w.sinks : 0;   // warps
    if (n_far + n_kv + n_q > 0x7fffffffLL || joins / 8 > 0x7ffffffeLL)
        return set_error(RA_ERR_UNSUPPORTED, "too many tiles for one launch");
    a.n_far = (int)n_far;
    a.n_kv = (int)n_kv;
    const int64_t rows = w.B * w.L * w.H, per_block = 8 * 4 * (256 / D);
    auto dot = o_bf16 ? bwd_window_dot<D, true> : bwd_window_dot<D, false>;
    auto kern = attn_bwd_window_kernel<D>;
    const int smem = (int)BwdWindowSmem<D>::kBytes;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return set_error(RA_ERR_CUDA, "cudaFuncSetAttribute(MaxDynamicSharedMemorySize) failed");
    if ((rows + per_block - 1) / per_block > 0x7fffffffLL)
        return set_error(RA_ERR_UNSUPPORTED, "too many rows for one launch");
    cudaError_t e = launch_dependent(dot, (unsigned)((rows + per_block - 1) / per_block), 256, 0, stream,
                                     static_cast<const uint16_t *>(dout), o,
                                     reinterpret_cast<float *>(workspace + space.dvec), rows, a.H, w.L);
    if (e == cudaSuccess)
        e = launch_dependent(kern, (unsigned)(n_far + n_kv + n_q), 384, smem, stream, mq, mk, mv, mdo, a);
    if (e == cudaSuccess && joins > 0)
        e = launch_dependent(bwd_sink_join<D>, (unsigned)((joins + 7) / 8), 256, 0, stream, a);
    return launched(e);
}

}  // namespace
}  // namespace ra

extern "C" {

ra_status ra_window_attn_fwd(const void *q, const void *k, const void *v, void *o, float *lse,
                             const int32_t *cu_seqlens, int n_seqs, int64_t B, int64_t L, int64_t H, int64_t H_kv,
                             int d, int64_t window, int64_t sinks, float scale, unsigned flags, void *workspace,
                             size_t workspace_bytes, void *stream) {
    using namespace ra;
    if (flags & ~RA_FLAG_O_BF16) return set_error(RA_ERR_INVALID_ARG, "unknown flag bits");
    Window w{B, L, H, H_kv, d, 0, 0, scale, nullptr, 0};
    const ra_status st = check(w, window, sinks, cu_seqlens, n_seqs);
    if (st != RA_OK) return st;
    if (B * L * H == 0) return RA_OK;
    const void *ptrs[] = {q, k, v, o, lse, workspace};
    for (const void *p : ptrs) {
        if (!p) return set_error(RA_ERR_INVALID_ARG, "null pointer argument");
        if (!aligned16(p)) return set_error(RA_ERR_ALIGNMENT, "every tensor pointer must be 16-byte aligned");
    }
    if (workspace_bytes < RA_WORKSPACE_MIN_BYTES)
        return set_error(RA_ERR_INVALID_ARG, "workspace smaller than RA_WORKSPACE_MIN_BYTES");
    unsigned *status = static_cast<unsigned *>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (few_keys(B, L, H, d, w.window, w.sinks)) {
        WindowFew f{};
        f.q = static_cast<const uint16_t *>(q);
        f.k = static_cast<const uint16_t *>(k);
        f.v = static_cast<const uint16_t *>(v);
        f.o = o;
        f.lse = lse;
        f.cu = w.cu;
        f.n_seqs = w.n_seqs;
        f.S = (int)L;
        f.H = (int)H;
        f.Hkv = (int)H_kv;
        f.window = w.window;
        f.sinks = w.sinks;
        f.scale_log2 = softmax_scale(w) * 1.4426950408889634f;
        return launch_window_few(f, d, (flags & RA_FLAG_O_BF16) != 0, B, s);
    }
    if (flags & RA_FLAG_O_BF16)
        return d == 128 ? launch_fwd<128, false>(w, q, k, v, o, lse, status, s)
                        : launch_fwd<64, false>(w, q, k, v, o, lse, status, s);
    return d == 128 ? launch_fwd<128, true>(w, q, k, v, o, lse, status, s)
                    : launch_fwd<64, true>(w, q, k, v, o, lse, status, s);
}

size_t ra_window_attn_bwd_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t H_kv, int d, int64_t window,
                                          int64_t sinks, int n_seqs) {
    if (B < 0 || L < 0 || H < 0 || H_kv < 0 || window < 1 || sinks < 0 || n_seqs < 0 || (d != 64 && d != 128)) return 0;
    if (B > (int64_t)1 << 20 || L > (int64_t)1 << 29 || H > (int64_t)1 << 20 || H_kv > H || n_seqs > ra::kMostSeqs) return 0;
    return ra::bwd_space(B, L, H, H_kv, d, window, sinks, n_seqs).total;
}

ra_status ra_window_attn_bwd(const void *q, const void *k, const void *v, const void *o, const void *dout,
                             const float *lse, void *dq, void *dk, void *dv, const int32_t *cu_seqlens, int n_seqs,
                             int64_t B, int64_t L, int64_t H, int64_t H_kv, int d, int64_t window, int64_t sinks,
                             float scale, unsigned flags, void *workspace, size_t workspace_bytes, void *stream) {
    using namespace ra;
    if (flags & ~(RA_FLAG_O_BF16 | RA_FLAG_GRAD_BF16)) return set_error(RA_ERR_INVALID_ARG, "unknown flag bits");
    Window w{B, L, H, H_kv, d, 0, 0, scale, nullptr, 0};
    const ra_status st = check(w, window, sinks, cu_seqlens, n_seqs);
    if (st != RA_OK) return st;
    if (B * L * H == 0) return RA_OK;
    const void *ptrs[] = {q, k, v, o, dout, lse, dq, dk, dv, workspace};
    for (const void *p : ptrs) {
        if (!p) return set_error(RA_ERR_INVALID_ARG, "null pointer argument");
        if (!aligned16(p)) return set_error(RA_ERR_ALIGNMENT, "every tensor pointer must be 16-byte aligned");
    }
    const BwdSpace space = bwd_space(B, L, H, H_kv, d, window, sinks, n_seqs);
    if (space.total == 0) return set_error(RA_ERR_UNSUPPORTED, "sizes beyond the supported range");
    if (workspace_bytes < space.total)
        return set_error(RA_ERR_INVALID_ARG, "workspace smaller than ra_window_attn_bwd_workspace_bytes()");
    auto launch = d == 128 ? launch_bwd<128> : launch_bwd<64>;
    return launch(w, q, k, v, o, (flags & RA_FLAG_O_BF16) != 0, dout, lse, dq, dk, dv,
                  (flags & RA_FLAG_GRAD_BF16) != 0, static_cast<uint8_t *>(workspace), space,
                  static_cast<cudaStream_t>(stream));
}

}  // extern "C"
