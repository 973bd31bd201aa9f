// attn_paged_few.cu -- paged attention of chunks over few keys: short prompts,
// or a short window.
//
// A CTA takes up to 64 rows (tokens by the query heads of one key/value head)
// of a sequence and copies the keys that they see to shared memory, as many as
// it has room for at a time; its four warps take 16 rows each through them, 16
// keys at a time (ra_warp_mma.cuh), each stopping at its own rows' last key.
// The tensor-core form pays about 7 us a CTA beside its 128-key tiles and pads a
// short sequence to 256 rows; where the two cross is written at few_keys
// (attn_paged.cu).  Bound by the latency of one pass: table, keys, at most eight
// dependent chunks, rows out.  40 prompts of 33-40 tokens, 8 / 8 heads, d = 64:
// 6.6 us against 17.5.
#include <cmath>

#include "paged_launch.h"
#include "ra_launch.h"
#include "ra_paged.cuh"
#include "ra_warp_mma.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4, kChunk = kPagedChunk, kMostChunks = 32;

struct FewArgs {
    PagedSeqs seqs;                 // unit_tokens: 64 / group
    const uint16_t *q, *k, *v;
    int64_t q_stride, page_stride;
    void *o;
    float *lse;
    float scale_log2;
    unsigned *status;
    int n_units, room;              // room: chunks in shared memory
};

// The chunks of rows whose first row has `first` and whose last key is
// last_hi - 1, as paged_chunks has them for a sequence.
__device__ __forceinline__ PagedChunks row_chunks(const RowKeys &first, int last_hi) {
    PagedChunks c{};
    c.m0 = first.lo / kChunk;
    const int m1 = (last_hi + kChunk - 1) / kChunk;
    if (first.shi > first.slo) c.n_sink = min((first.shi + kChunk - 1) / kChunk, c.m0);
    c.count = c.n_sink + max(m1 - c.m0, 0);
    return c;
}

template <int D, bool O_BF16>
__global__ void __launch_bounds__(32 * kWarps, D == 64 ? 3 : 2) paged_few_kernel(const FewArgs a) {
    constexpr int KS = D / 16, CPR = D / 8;
    constexpr uint32_t kHalf = kChunk * D * 2;       // a chunk's keys
    constexpr int kOut = D * 2 + 16;                 // bytes of a staged bf16 row
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int ids[kMostChunks];
    const PagedSeqs &sq = a.seqs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    pdl_wait();
    // blockIdx.x = hk * units + unit
    const int unit = blockIdx.x % a.n_units, hk = blockIdx.x / a.n_units;
    const int s = paged_find_seq(sq, unit);
    const PagedUnit u = paged_unit(sq, s, unit - paged_first_unit(sq, s));
    if (hk == 0 && u.first == 0 && threadIdx.x == 0 && paged_bad_counts(sq, s)) atomicOr(a.status, RA_DEV_PAGE_BIT);
    if (u.n <= 0) return;
    const int rows = u.n * sq.group;
    const PagedChunks all = row_chunks(paged_row(sq, u.p0), u.p0 + u.n);
    const uint32_t keys = smem_u32(smem), values = keys + a.room * kHalf;

    // this warp's rows
    const int w0 = warp * 16;
    const bool any = w0 < rows;
    WarpRows<D, 1> rw;
    rw.clear();
    int pos[2], tok[2], head[2];
    PagedChunks mine{};
    int all_lo = 0, all_hi = 0, all_shi = 0;
    if (any) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = min(w0 + 8 * h + g, rows - 1);
            tok[h] = r / sq.group;
            head[h] = hk * sq.group + r - tok[h] * sq.group;
            pos[h] = u.p0 + tok[h];
            const uint16_t *src = a.q + (size_t)(u.t0 + tok[h]) * a.q_stride + (size_t)head[h] * D + 2 * t4;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                rw.q[0][ks][h] = *reinterpret_cast<const uint32_t *>(src + ks * 16);
                rw.q[0][ks][2 + h] = *reinterpret_cast<const uint32_t *>(src + ks * 16 + 8);
            }
        }
        const int p_first = u.p0 + w0 / sq.group, p_last = u.p0 + (min(w0 + 16, rows) - 1) / sq.group;
        const RowKeys first = paged_row(sq, p_first), last = paged_row(sq, p_last);
        mine = row_chunks(first, p_last + 1);
        // chunks inside [all_lo, all_hi) or [0, all_shi) are seen whole by every row
        all_lo = last.lo, all_hi = first.hi, all_shi = first.shi > first.slo ? first.shi : 0;
    }
    // chunk number of `all` that holds chunk c of the warp's list: the warp's
    // sinks are the unit's or lie among its main keys
    int c = 0;
    auto key_of = [&](const PagedChunks &l, int i) { return paged_chunk_key(l, i); };
    auto place = [&](int k0) { return k0 >= all.m0 * kChunk ? all.n_sink + k0 / kChunk - all.m0 : k0 / kChunk; };

    for (int base = 0; base < all.count; base += a.room) {
        const int n = min(a.room, all.count - base);
        if (base > 0) __syncthreads();      // the chunks before have been read
        if ((int)threadIdx.x < n) {
            const int k0 = key_of(all, base + threadIdx.x);
            int id = -1;
            if (k0 < u.len) {
                id = sq.table[(size_t)s * sq.max_pages + k0 / sq.page];
                if ((unsigned)id >= (unsigned)sq.n_pages) {
                    atomicOr(a.status, RA_DEV_PAGE_BIT);
                    id = -1;
                }
            }
            ids[threadIdx.x] = id;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < n * kChunk * CPR; e += 32 * kWarps) {
            const int row = e / CPR, pc = e % CPR;
            const int key = key_of(all, base + row / kChunk) + row % kChunk, id = ids[row / kChunk];
            const bool in = id >= 0 && key < u.len;
            const size_t at = in ? (size_t)id * a.page_stride + ((size_t)(key & (sq.page - 1)) * sq.Hkv + hk) * D + pc * 8 : 0;
            const uint32_t to = row * (D * 2) + ((pc ^ (row & 7)) << 4);
            cp_async16(keys + to, a.k + at, in);
            cp_async16(values + to, a.v + at, in);
        }
        cp_async_commit();
        cp_async_wait<0>();
        __syncthreads();
        for (; any && c < mine.count; ++c) {
            const int k0 = key_of(mine, c), at = place(k0) - base;
            if (at >= n) break;
            if (at < 0) continue;
            const bool whole = (k0 >= all_lo && k0 + kChunk <= all_hi) || k0 + kChunk <= all_shi;
            rw.chunk(keys + at * kHalf, values + at * kHalf, a.scale_log2, whole, lane, [&](int, int h) {
                const RowKeys rk = paged_row(sq, pos[h]);
                return seen_bits(rk.lo, rk.hi, rk.slo, rk.shi, k0);
            });
        }
    }
    if (!any) return;
    uint8_t *stage = smem + 2 * a.room * kHalf + warp * 16 * kOut;
    int64_t at = -1;       // the row's first element, in the lane that has the row's number
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float l = rw.l[0][h];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const int r = w0 + 8 * h + g;
        const size_t row = ((size_t)(u.t0 + tok[h]) * sq.H + head[h]) * D;
        if (t4 == 0 && r < rows && a.lse)
            a.lse[(size_t)head[h] * sq.T + u.t0 + tok[h]] = l > 0.f ? (rw.m[0][h] + lg2(l)) * 0.6931471805599453f : -INFINITY;
        if constexpr (O_BF16) {
            uint32_t *dst = reinterpret_cast<uint32_t *>(stage + (8 * h + g) * kOut) + t4;
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
                dst[n * 4] = pack_bf16x2(rw.acc[0][n][2 * h] * inv, rw.acc[0][n][2 * h + 1] * inv);
        } else if (r < rows) {
            float *dst = static_cast<float *>(a.o) + row + 2 * t4;
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
                *reinterpret_cast<float2 *>(dst + n * 8) = make_float2(rw.acc[0][n][2 * h] * inv, rw.acc[0][n][2 * h + 1] * inv);
        }
    }
    if constexpr (O_BF16) {
        if (lane < 16 && w0 + lane < rows) {
            const int r = w0 + lane, tk = r / sq.group;
            at = (int64_t)(((size_t)(u.t0 + tk) * sq.H + hk * sq.group + r - tk * sq.group) * D);
        }
        __syncwarp();
#pragma unroll
        for (int e = lane; e < 16 * CPR; e += 32) {
            const int r = e / CPR, pc = e % CPR;
            const long long dst = __shfl_sync(0xffffffffu, (long long)at, r);
            if (dst >= 0)
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o) + dst + pc * 8) =
                    *reinterpret_cast<const uint4 *>(stage + r * kOut + pc * 16);
        }
    }
}

}  // namespace

ra_status launch_paged_few(const PagedFewLaunch &t, cudaStream_t stream) {
    FewArgs a{};
    a.seqs = t.seqs;
    a.q = static_cast<const uint16_t *>(t.q);
    a.k = static_cast<const uint16_t *>(t.k);
    a.v = static_cast<const uint16_t *>(t.v);
    a.q_stride = t.q_stride;
    a.page_stride = t.page_stride;
    a.o = t.o;
    a.lse = t.lse;
    a.scale_log2 = t.scale_log2;
    a.status = t.status;
    a.n_units = t.units;
    // room for the keys the call expects; longer lists take turns
    const int64_t want = (t.keys + kChunk - 1) / kChunk + 2;
    a.room = (int)(want < kPagedFewRoom ? want : kPagedFewRoom);
    static_assert(kPagedFewRoom <= kMostChunks, "a thread and a place for each chunk's page");
    auto smem_of = [&](int room) { return (size_t)room * 2 * kChunk * t.d * 2 + kWarps * 16 * (t.d * 2 + 16); };
    const size_t smem = smem_of(a.room), most = smem_of(kPagedFewRoom);
    auto kern = t.d == 128 ? (t.o_bf16 ? paged_few_kernel<128, true> : paged_few_kernel<128, false>)
                           : (t.o_bf16 ? paged_few_kernel<64, true> : paged_few_kernel<64, false>);
    // the limit is the form's largest, not this call's: host threads share it
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) != cudaSuccess)
        return set_error(RA_ERR_CUDA, "cudaFuncSetAttribute(MaxDynamicSharedMemorySize) failed");
    const int64_t grid = (int64_t)t.units * t.seqs.Hkv;
    if (grid > 0x7fffffffLL) return set_error(RA_ERR_UNSUPPORTED, "too many query tiles for one launch");
    return launched(launch_dependent(kern, (unsigned)grid, 32 * kWarps, smem, stream, a));
}

}  // namespace ra
