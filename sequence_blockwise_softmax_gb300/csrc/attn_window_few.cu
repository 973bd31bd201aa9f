// attn_window_few.cu -- the windowed forward where a row sees few keys.
//
// A CTA takes 64 tokens of one key/value head, copies the keys and values that
// they see -- at most 64 + window + sinks tokens -- to shared memory once, and
// its four warps take 16 rows of one query head after another through them, 16
// keys at a time (ra_warp_mma.cuh): a row block meets window / 16 + 2 chunks and
// the one or more that hold the sinks, instead of whole 128-key tiles.  There
// is no pipeline inside a CTA; two or more CTAs on an SM cover one another's
// loads.  Where there are few rows a CTA takes 16 of one head, and its warps
// share their keys and join: the chain of a warp's chunks, 0.2 us each, is a
// quarter as long.  512 tokens, 2 heads, d = 64: window 128: 6.0 -> 4.1 us, 400:
// 8.0 (tensor-core form) -> 6.0.
//
// The tensor-core form (attn_fwd_kernel.cuh) costs about 7 us a CTA of 256 rows
// beside its tiles, which at these sizes is most of its time; where the two cross
// is written at few_keys (attn_window.cu).  With many tokens this form is bound by
// the CTAs an SM holds (two at d = 128, three at d = 64, by registers and shared
// memory) and each one's latencies: 40000 tokens, 16 / 8 heads, window 16: 80 us
// at d = 64 and 142 at d = 128, where the bytes take 36 and 72.
#include <cmath>
#include <type_traits>

#include "ra_launch.h"
#include "ra_warp_mma.cuh"
#include "ra_window.cuh"
#include "window_few.h"

namespace ra {
namespace {

constexpr int kWarps = 4, kChunk = 16;
// rows of a CTA: 16 a warp, or 16 whose keys the warps share
constexpr int few_rows(bool split) { return split ? 16 : 16 * kWarps; }

// The chunks of a block of rows, as range_walk has tiles: n_sink from key s0 on,
// then from m0 on (both multiples of 16).
struct FewChunks {
    int s0, n_sink, m0, count;
    __device__ int key(int c) const { return c < n_sink ? s0 + c * kChunk : m0 + (c - n_sink) * kChunk; }
};
__device__ __forceinline__ FewChunks few_chunks(const RowKeys &first, int last_hi) {
    FewChunks c;
    c.m0 = first.lo & ~(kChunk - 1);
    c.s0 = first.slo & ~(kChunk - 1);
    const int s1 = min(first.shi, c.m0);
    c.n_sink = first.shi > first.slo && s1 > c.s0 ? (s1 - c.s0 + kChunk - 1) / kChunk : 0;
    c.count = c.n_sink + (last_hi - c.m0 + kChunk - 1) / kChunk;
    return c;
}

// SPLIT: the warps take the chunks of the CTA's 16 rows in turn and join at the end.
template <int D, bool O_BF16, bool SPLIT>
__global__ void __launch_bounds__(32 * kWarps, D == 64 ? 3 : 2) window_few_kernel(const WindowFew a) {
    constexpr int KS = D / 16, CPR = D / 8, kRows = few_rows(SPLIT), kJoin = D + 8;   // kJoin: floats per row of the join
    __shared__ float s_m[kWarps][16], s_l[kWarps][16];
    constexpr uint32_t kHalf = kChunk * D * 2;       // a chunk's keys
    constexpr int kOut = D * 2 + 16;                 // bytes of a staged bf16 row
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int group = a.H / a.Hkv;
    pdl_wait();
    const int S = packed_tokens(a.cu, a.n_seqs, a.S);     // rows behind them are left alone
    // blockIdx.x = ((b * H_kv + hk) * parts of the group + part) * blocks + block
    const int blk = blockIdx.x % a.blocks;
    int rest = blockIdx.x / a.blocks;
    const int head0 = rest % a.group_parts * a.heads, head1 = min(group, head0 + a.heads);
    rest /= a.group_parts;
    const int hk = rest % a.Hkv, b = rest / a.Hkv;
    const int r0 = blk * kRows, r_end = min(S, r0 + kRows);
    if (r0 >= S) return;
    const FewChunks all = few_chunks(window_row(a.cu, a.n_seqs, S, r0, a.window, a.sinks), r_end);
    // a call's own bound on its chunks; only boundaries that do not increase could pass it
    const int n_chunks = min(all.count, a.max_chunks);
    const uint32_t keys = smem_u32(smem), values = keys + a.max_chunks * kHalf;
    {
        // the tokens' rows of head hk: 16-byte pieces, a token's pieces to neighbouring threads
        const size_t head = ((size_t)b * a.S * a.Hkv + hk) * D;
        for (int e = threadIdx.x; e < n_chunks * kChunk * CPR; e += 32 * kWarps) {
            const int row = e / CPR, pc = e % CPR;
            const int key = all.key(row / kChunk) + row % kChunk;
            const bool in = key < S;
            const size_t at = in ? head + (size_t)key * a.Hkv * D + pc * 8 : 0;
            const uint32_t to = row * (D * 2) + ((pc ^ (row & 7)) << 4);
            cp_async16(keys + to, a.k + at, in);
            cp_async16(values + to, a.v + at, in);
        }
        cp_async_commit();
    }
    // this warp's 16 rows and their chunks
    const int w0 = SPLIT ? r0 : r0 + warp * 16, w_end = min(S, w0 + 16);
    const bool any = w0 < S;
    RowKeys rk[2];
    FewChunks mine{};
    RowKeys first{};
    if (any) {
        first = window_row(a.cu, a.n_seqs, S, w0, a.window, a.sinks);
        mine = few_chunks(first, w_end);
#pragma unroll
        for (int h = 0; h < 2; ++h) rk[h] = window_row(a.cu, a.n_seqs, S, min(w0 + 8 * h + g, S - 1), a.window, a.sinks);
    }
    // keys that every row of the warp sees: [all_lo, first.hi)
    const int all_lo = (int)__reduce_max_sync(0xffffffffu, (unsigned)max(any ? rk[0].lo : 0, any ? rk[1].lo : 0));
    uint8_t *stage = smem + 2 * a.max_chunks * kHalf + warp * 16 * kOut;
    auto load_q = [&](uint32_t (&q)[KS][4], int hq) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = w0 + 8 * h + g;
            const uint16_t *src = a.q + (((size_t)b * a.S + min(r, S - 1)) * a.H + hq) * D + 2 * t4;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                q[ks][h] = *reinterpret_cast<const uint32_t *>(src + ks * 16);
                q[ks][2 + h] = *reinterpret_cast<const uint32_t *>(src + ks * 16 + 8);
            }
        }
    };
    WarpRows<D, 1> rw;
    if (any) load_q(rw.q[0], hk * group + head0);
    for (int head = head0; head < head1; ++head) {
        const int hq = hk * group + head;
        rw.clear();
        if (head == head0) {
            cp_async_wait<0>();
            __syncthreads();
        }
        if (!any) continue;
        for (int c = SPLIT ? warp : 0; c < mine.count; c += SPLIT ? kWarps : 1) {
            const int k0 = mine.key(c);
            // its place in shared memory: among the main keys, or the sinks before them
            const int at = k0 >= all.m0 ? all.n_sink + (k0 - all.m0) / kChunk : (k0 - all.s0) / kChunk;
            if ((unsigned)at >= (unsigned)n_chunks) continue;
            const bool whole = k0 >= all_lo && k0 + kChunk <= first.hi;
            rw.chunk(keys + at * kHalf, values + at * kHalf, a.scale_log2, whole, lane,
                     [&](int, int h) { return seen_bits(rk[h].lo, rk[h].hi, rk[h].slo, rk[h].shi, k0); });
        }
        if (head + 1 < head1) load_q(rw.q[0], hq + 1);     // on its way while the rows are written
        if constexpr (SPLIT) {
            // (any holds for every warp or for none: the rows are the CTA's)
            float *rows = reinterpret_cast<float *>(smem + 2 * a.max_chunks * kHalf);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                rw.l[0][h] += __shfl_xor_sync(0xffffffffu, rw.l[0][h], 1);
                rw.l[0][h] += __shfl_xor_sync(0xffffffffu, rw.l[0][h], 2);
                if (t4 == 0) {
                    s_m[warp][8 * h + g] = rw.m[0][h];
                    s_l[warp][8 * h + g] = rw.l[0][h];
                }
            }
            __syncthreads();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = 8 * h + g;
                const float top = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
                const float f = rw.m[0][h] > -INFINITY ? ex2(rw.m[0][h] - top) : 0.f;
                float *dst = rows + ((size_t)warp * 16 + r) * kJoin + 2 * t4;
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *reinterpret_cast<float2 *>(dst + n * 8) = make_float2(rw.acc[0][n][2 * h] * f, rw.acc[0][n][2 * h + 1] * f);
            }
            __syncthreads();
            for (int e = threadIdx.x; e < 16 * (D / 4); e += 32 * kWarps) {
                const int r = e / (D / 4), col = (e % (D / 4)) * 4;
                if (w0 + r >= S) break;
                float x[4] = {}, top = -INFINITY, l = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float4 f = *reinterpret_cast<const float4 *>(rows + ((size_t)w * 16 + r) * kJoin + col);
                    x[0] += f.x, x[1] += f.y, x[2] += f.z, x[3] += f.w;
                    top = fmaxf(top, s_m[w][r]);
                }
#pragma unroll
                for (int w = 0; w < kWarps; ++w) l += s_m[w][r] > -INFINITY ? s_l[w][r] * ex2(s_m[w][r] - top) : 0.f;
                const float inv = l > 0.f ? 1.f / l : 0.f;
                const size_t at = (((size_t)b * a.S + w0 + r) * a.H + hq) * D + col;
                if constexpr (O_BF16)
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.o) + at) =
                        make_uint2(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv));
                else
                    *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + at) =
                        make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
                if (col == 0)
                    a.lse[((size_t)b * a.H + hq) * a.S + w0 + r] = l > 0.f ? (top + lg2(l)) * 0.6931471805599453f : -INFINITY;
            }
            __syncthreads();     // before the next head's rows
            continue;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float l = rw.l[0][h];
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const int r = w0 + 8 * h + g;
            if (t4 == 0 && r < S)
                a.lse[((size_t)b * a.H + hq) * a.S + r] = l > 0.f ? (rw.m[0][h] + lg2(l)) * 0.6931471805599453f : -INFINITY;
            if constexpr (O_BF16) {
                uint32_t *row = reinterpret_cast<uint32_t *>(stage + (8 * h + g) * kOut) + t4;
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    row[n * 4] = pack_bf16x2(rw.acc[0][n][2 * h] * inv, rw.acc[0][n][2 * h + 1] * inv);
            } else if (r < S) {
                float *row = static_cast<float *>(a.o) + (((size_t)b * a.S + r) * a.H + hq) * D + 2 * t4;
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *reinterpret_cast<float2 *>(row + n * 8) = make_float2(rw.acc[0][n][2 * h] * inv, rw.acc[0][n][2 * h + 1] * inv);
            }
        }
        if constexpr (O_BF16) {
            __syncwarp();
#pragma unroll
            for (int e = lane; e < 16 * CPR; e += 32) {
                const int r = e / CPR, pc = e % CPR;
                if (w0 + r < S)
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o) + (((size_t)b * a.S + w0 + r) * a.H + hq) * D + pc * 8) =
                        *reinterpret_cast<const uint4 *>(stage + r * kOut + pc * 16);
            }
            __syncwarp();
        }
    }
}

}  // namespace

bool window_few_split(int64_t B, int64_t S, int64_t H, int d, int window, int sinks) {
    const int chunks = window_few_chunks((int)S, window, sinks, true);
    const size_t smem = window_few_smem(chunks, d, true), most = (size_t)227 << 10;
    const int per_sm = d == 64 && 2 * (smem + 1024) <= most + 1024 ? 2 : 1;
    return chunks > 2 && smem <= kWindowFewSmem && B * H * ((S + 15) / 16) <= 152 * per_sm;
}

int window_few_chunks(int S, int window, int sinks, bool split) {
    const int kRows = few_rows(split);
    // The main keys end at the rows' end, a multiple of 16 (or of the tokens),
    // and begin window - 1 before the first row, earlier by up to `sinks` where
    // the sinks touch the window; else the sinks lie apart, anywhere.
    auto chunks = [](int64_t keys) { return (keys + kChunk - 1) / kChunk; };
    const int64_t main = chunks(kRows + (int64_t)window - 1), touching = chunks(kRows + (int64_t)window - 1 + sinks);
    const int64_t apart = main + (sinks > 0 ? chunks(sinks + kChunk - 1) : 0);
    const int64_t most = chunks(S), need = touching > apart ? touching : apart;
    return (int)(need < most ? need : most);
}

size_t window_few_smem(int chunks, int d, bool split) {
    return (size_t)chunks * 2 * kChunk * d * 2 + kWarps * 16 * (split ? (d + 8) * 4 : d * 2 + 16);
}

ra_status launch_window_few(WindowFew a, int d, bool o_bf16, int64_t B, cudaStream_t stream) {
    const bool split = window_few_split(B, a.S, a.H, d, a.window, a.sinks);
    a.blocks = (a.S + few_rows(split) - 1) / few_rows(split);
    a.max_chunks = window_few_chunks(a.S, a.window, a.sinks, split);
    const size_t smem = window_few_smem(a.max_chunks, d, split);
    auto pick = [&](auto s) {
        constexpr bool SPLIT = decltype(s)::value;
        return d == 128 ? (o_bf16 ? window_few_kernel<128, true, SPLIT> : window_few_kernel<128, false, SPLIT>)
                        : (o_bf16 ? window_few_kernel<64, true, SPLIT> : window_few_kernel<64, false, SPLIT>);
    };
    auto kern = split ? pick(std::true_type()) : pick(std::false_type());
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kWindowFewSmem) != cudaSuccess)
        return set_error(RA_ERR_CUDA, "cudaFuncSetAttribute(MaxDynamicSharedMemorySize) failed");
    // a CTA takes the heads of a group one after another; where there are too
    // few CTAs for that, each takes fewer and the keys are copied again
    const int group = a.H / a.Hkv;
    const int64_t whole = (int64_t)a.blocks * a.Hkv * B;
    const int64_t parts = whole >= 304 ? 1 : (304 + whole - 1) / whole;
    a.heads = (int)(parts >= group ? 1 : (group + parts - 1) / parts);
    a.group_parts = (group + a.heads - 1) / a.heads;
    const int64_t grid = whole * a.group_parts;
    if (grid > 0x7fffffffLL) return set_error(RA_ERR_UNSUPPORTED, "too many query tiles for one launch");
    return launched(launch_dependent(kern, (unsigned)grid, 32 * kWarps, smem, stream, a));
}

}  // namespace ra
