// attn_paged_tokens.cu -- paged attention of few rows: single tokens, or a few
// tokens of each sequence, up to 32 rows (tokens x query heads) per key/value
// head.
//
// Bound by the cache's bytes: each key and value is used by a handful of rows,
// so the kernel is a stream of loads with small products beside it.  The work
// is one flat list of 16-key chunks -- sequence by sequence, key/value head by
// head, key by key -- cut into equal runs, one per CTA (two CTAs per SM): a
// batch of very different lengths leaves no CTA with more than its share, and
// one long sequence is spread over the whole GPU.  With few (sequence, head)
// pairs each pair is cut into pieces of its own instead, so that no CTA meets
// two of them and pays the end of a pair (about 3 us) twice.  A piece that is
// not a whole pair leaves O (unnormalised, fp32), the reference and the sum of
// exponentials in the workspace, and the CTA that counts the last piece of a
// pair adds them in the order of their keys, so the result does not depend on
// which one it is.  Up to 152 pairs that are not too long take no such way through
// memory: each pair gets a cluster of 2 to 16 CTAs, which join their equal pieces
// through shared memory (paged_tokens_cluster): one sequence of 1000 keys 7.4 -> 5.9
// us, 8 of 500-1000 10.3 -> 8.6.
//
// Inside a run the four warps take the chunks in turn and share nothing until
// the end of a head: each has its own ring of cp.async stages (96 KB per CTA in
// flight), its own m, l and O.  mma.sync m16n8k16 with the rows padded to 16:
// at 6.8 TB/s an SM sees a chunk (8 KB at d = 128) every 0.18 us and needs 48
// such products for it, a few per cent of the pipe, so the tensor pipe is not
// what bounds this; 128-row tcgen05 tiles would spend their time on padding.
// P enters its product as the sum of two bf16 values (ra_warp_mma.cuh), which
// costs a second product and leaves the output's own rounding as the only one.
//
// The mathematics: S = q K^T, P = 2^(S scale log2 e - m), l = sum P, O = P V / l,
// LSE = (m + log2 l) ln 2, with m moved rarely; pieces with (m_i, l_i, O_i) add to
// m = max m_i, l = sum l_i 2^(m_i - m), O = sum O_i 2^(m_i - m).
//
// Measured on a GB300, 32 / 8 heads, d = 128: 64 sequences of 200-16000 keys 362
// us (6.6 TB/s; the bytes alone take 353 at the copy rate), 8 of 3000-4000 keys
// 25 us, one of 1000 keys 6.1 us, which is a chain of latencies: lengths, table,
// keys, the warps' rows, the join.
#include <atomic>
#include <cmath>
#include <type_traits>

#include "paged_launch.h"
#include "ra_launch.h"
#include "ra_device.cuh"
#include "ra_paged.cuh"
#include "ra_warp_mma.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4;
constexpr int kChunk = kPagedChunk;

struct TokensArgs {
    PagedSeqs seqs;
    const uint16_t *q, *k, *v;
    int64_t q_stride, page_stride;  // elements
    void *o;
    float *lse;
    int o_bf16, whole_pairs;
    float scale_log2;
    unsigned *status;
    unsigned long long call;        // the call's tag, another one for every call of the process
    unsigned long long *counters;   // one per CTA: a call's tag, then the pieces counted in it
    float *part_o, *part_ml;        // [2 * CTAs, 16 * MT, d], [2 * CTAs, 16 * MT, 2]
};

template <int D>
struct TokensSmem {
    static constexpr int kStages = 384 / D;                       // 3 at d = 128, 6 at d = 64
    static constexpr uint32_t kHalf = kChunk * D * 2;             // a chunk's keys; its values follow
    static constexpr uint32_t kStage = 2 * kHalf;
    static constexpr uint32_t kWarp = kStages * kStage;
    static constexpr uint32_t kBytes = kWarps * kWarp;            // 96 KB
    static constexpr int kRow = D + 8;                            // floats per row of the warps' O at the end
};

// A pair's pieces are counted in the low bits of a word whose others are the
// call's tag, so that whatever other calls left in the workspace counts as
// nothing; the block that counts the last piece sets the word back to the tag
// and no pieces, where a replay of the same call begins.  A tag's upper half
// is, as fp32, a signalling NaN, which no arithmetic leaves behind: floats that
// other entry points keep in a workspace are never taken for a call's count.
constexpr unsigned long long kCountMask = 1023, kTag = 0xffaull << 52;
static_assert(kPagedTokensCtas <= (int)kCountMask, "a word counts as many pieces");
__host__ __device__ constexpr unsigned long long call_tag(unsigned long long n) { return kTag | ((n << 10) & ~(0xfffull << 52)); }

__device__ __forceinline__ unsigned long long swap_word(unsigned long long *word, unsigned long long old,
                                                        unsigned long long now) {
    unsigned long long seen;
    asm volatile("atom.cas.acq_rel.gpu.global.b64 %0, [%1], %2, %3;" : "=l"(seen) : "l"(word), "l"(old), "l"(now) : "memory");
    return seen;
}
// A block starts its own word (that of the pair whose first piece it may have)
// as early as it can, so that later counts find the call's tag there.
__device__ __forceinline__ void start_word(unsigned long long *word, unsigned long long call) {
    const unsigned long long old = *reinterpret_cast<volatile unsigned long long *>(word);
    if ((old & ~kCountMask) != call) swap_word(word, old, call);
}
// How many pieces were counted in this word before this one: one add where the
// word has the call's tag.  Where it has not, the add fell on what will be
// replaced; whoever replaces it counts itself, the others add again.
__device__ __forceinline__ int count_piece(unsigned long long *word, unsigned long long call) {
    while (true) {
        unsigned long long old;
        asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], 1;" : "=l"(old) : "l"(word) : "memory");
        if ((old & ~kCountMask) == call) return (int)(old & kCountMask);
        unsigned long long seen = *reinterpret_cast<volatile unsigned long long *>(word);
        while ((seen & ~kCountMask) != call) {
            old = seen;
            seen = swap_word(word, old, call + 1);
            if (seen == old) return 0;
        }
    }
}

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 x;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(addr) : "memory");
    return x;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
    float2 x;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(addr) : "memory");
    return x;
}
// `addr` in the shared memory of the cluster's CTA number `rank`
__device__ __forceinline__ uint32_t in_cluster(uint32_t addr, int rank) {
    uint32_t x;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(x) : "r"(addr), "r"(rank));
    return x;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// CLUSTER > 0: each pair's keys are cut into CLUSTER equal pieces (some maybe
// empty), which the CTAs of a cluster take and join through shared memory.
template <int D, int MT, int CLUSTER>
__global__ void __launch_bounds__(32 * kWarps, 2) paged_tokens_kernel(const TokensArgs a) {
    using L = TokensSmem<D>;
    constexpr int NS = L::kStages, KS = D / 16, CPR = D / 8;   // k-steps, 16-byte pieces per row
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ unsigned long long s_sum[kWarps];
    __shared__ long long s_at;                 // the first chunk (or piece) inside its sequence
    __shared__ PagedChunks s_list;
    __shared__ int s_seq, s_last;
    __shared__ float s_m[kWarps][16 * MT], s_l[kWarps][16 * MT];
    __shared__ float2 s_ml[16 * MT];           // CLUSTER: of the CTA's rows
    const PagedSeqs &sq = a.seqs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x;
    pdl_wait();

    // ---- how the work is cut, from the lengths the call finds
    // An inclusive scan of x over the block (its total added to `base`).
    auto scan = [&](unsigned long long x, unsigned long long &base) -> unsigned long long {
        unsigned long long inc = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long up = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += up;
        }
        __syncthreads();
        if (lane == 31) s_sum[warp] = inc;
        __syncthreads();
        inc += base;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) inc += s_sum[w];
            base += s_sum[w];
        }
        return inc;
    };
    const int blocks = (sq.n_seqs + blockDim.x - 1) / blockDim.x;    // of sequences, one to a thread
    const PagedChunks none{};
    auto list_of = [&](int s) { return s < sq.n_seqs ? paged_chunks(sq, s) : none; };
    PagedChunks mine = list_of(threadIdx.x);
    unsigned long long sum = 0;
    for (int i = 0; CLUSTER == 0 && i < blocks; ++i) {
        const PagedChunks l = i == 0 ? mine : list_of(i * blockDim.x + threadIdx.x);
        scan(paged_tally(l.count), sum);
    }
    // (sequence, head) pairs with new tokens, and their chunks
    const long long pairs = paged_tally_seqs(sum) * sq.Hkv;
    const long long total = paged_tally_chunks(sum) * sq.Hkv;
    const int grid = gridDim.x;
    // Few pairs: each is cut into pieces of its own, at most one to a CTA.
    // Many: equal runs of the flat list, whose ends fall anywhere.  Between half
    // as many pairs as CTAs and a third, by the length of a run: 128 pairs of
    // 14400-16000 keys 152 us in runs and 180 in pieces, of 16-4000 41 and 28.
    const bool flat = CLUSTER == 0 && !a.whole_pairs && (pairs * 2 > grid || (pairs * 3 > grid && total > 96ll * grid));
    const long long room = flat ? grid : max(grid - pairs, 1ll);
    const long long per64 = total < 0x7fffffff ? (long long)(((unsigned)total + (unsigned)room - 1) / (unsigned)room)
                                               : (total + room - 1) / room;
    // A piece of n chunks costs its CTA about 0.09 n us, each piece its pair's
    // join about 0.07 us: n is at least the square root that balances them.
    const int balanced = (int)sqrtf(0.8f * (float)total / (float)(pairs > 0 ? pairs : 1));
    int per = max((int)per64, max(balanced, kPagedMinRun));
    if (a.whole_pairs) per = 0x3fffffff;       // one CTA to a pair
    if (cta == 0) {
        for (int s = threadIdx.x; s < sq.n_seqs; s += blockDim.x)
            if (paged_bad_counts(sq, s)) atomicOr(a.status, RA_DEV_PAGE_BIT);
    }
    // where this CTA begins: chunk (or piece) number `at` of the list
    const long long at = flat ? (long long)cta * per : cta;
    {
        unsigned long long base = 0;
        for (int i = 0; i < blocks; ++i) {
            if (i > 0) mine = list_of(i * blockDim.x + threadIdx.x);
            const int pieces = CLUSTER ? (mine.count > 0 ? CLUSTER : 0) : (mine.count + per - 1) / per;
            const long long n = (long long)(flat ? mine.count : pieces) * sq.Hkv;
            const long long inc = (long long)scan(n, base);
            if (n > 0 && inc - n <= at && at < inc) {
                s_seq = i * blockDim.x + threadIdx.x;
                s_list = mine;
                s_at = at - (inc - n);
            }
            if ((long long)base > at) break;
        }
        if (at >= (long long)base) return;
    }
    __syncthreads();
    int seq = s_seq;
    PagedChunks cl = s_list;
    int hk, c_at, first_cta = 0, last_cta = 0;
    long long pos = at;
    const long long end = at + per < total ? at + per : total;    // of a flat run
    {
        if constexpr (CLUSTER > 0) per = (cl.count + CLUSTER - 1) / CLUSTER;
        const unsigned each = flat ? cl.count : CLUSTER ? CLUSTER : (cl.count + per - 1) / per;
        hk = s_at < 0x7fffffff ? (int)((unsigned)s_at / each) : (int)(s_at / each);
        const int in = (int)(s_at - (long long)hk * each);
        c_at = flat ? in : min(in * per, cl.count);
        first_cta = cta - in;             // of a pair in pieces
        last_cta = first_cta + (int)each - 1;
    }

    const uint32_t ring = smem_u32(smem) + warp * L::kWarp;
    const int g = lane >> 2, t4 = lane & 3;
    bool word_started = CLUSTER > 0 || a.whole_pairs;      // no pair is cut, no word is used (and there may be more CTAs than words)

    // ---- one head's keys (or this run's part of them) after another
    while (true) {
        const long long unit_begin = pos - c_at, unit_end = unit_begin + cl.count;
        const int c_end = flat ? (int)(unit_end < end ? cl.count : end - unit_begin) : (int)min((long long)cl.count, (long long)c_at + per);
        const int rows = cl.n * sq.group;

        // chunks inside [all_lo, all_hi) or [0, all_shi) are seen whole by every row
        const RowKeys first = paged_row(sq, cl.p0), last = paged_row(sq, cl.p0 + cl.n - 1);
        const int all_lo = last.lo, all_hi = first.hi, all_shi = first.shi > first.slo ? first.shi : 0;

        auto key_of = [&](int c) { return paged_chunk_key(cl, c); };
        const int *row_table = sq.table + (size_t)seq * sq.max_pages;
        auto page_of = [&](int c) -> int {
            const int k0 = key_of(c);
            return c < c_end && k0 < cl.len ? row_table[k0 / sq.page] : 0;
        };
        // load chunk c (of page id) into its stage; every call commits one group
        auto load = [&](int c, int stage, int id) {
            if (c < c_end) {
                const int k0 = key_of(c);
                bool ok = k0 < cl.len;
                if (ok && (unsigned)id >= (unsigned)sq.n_pages) {
                    ok = false;
                    if (lane == 0) atomicOr(a.status, RA_DEV_PAGE_BIT);
                }
                const size_t off = ok ? (size_t)id * a.page_stride + ((size_t)(k0 & (sq.page - 1)) * sq.Hkv + hk) * D : 0;
                const uint32_t dst = ring + stage * L::kStage;
                constexpr int ROWS = 32 / CPR;       // keys per pass of the warp
                const int key = lane / CPR, pc = lane % CPR;
#pragma unroll
                for (int i = 0; i < kChunk / ROWS; ++i) {
                    const int kk = i * ROWS + key;
                    const bool in = ok && k0 + kk < cl.len;
                    const size_t at = in ? off + (size_t)kk * sq.Hkv * D + pc * 8 : 0;
                    const uint32_t to = dst + kk * (D * 2) + ((pc ^ (kk & 7)) << 4);
                    cp_async16(to, a.k + at, in);
                    cp_async16(to + L::kHalf, a.v + at, in);
                }
            }
            cp_async_commit();
        };

        int c = c_at + warp;
        int next_id = page_of(c);
#pragma unroll
        for (int s = 0; s < NS - 1; ++s) {
            const int id = next_id;
            next_id = page_of(c + (s + 1) * kWarps);
            load(c + s * kWarps, s, id);
        }
        if (!word_started && threadIdx.x == 32 * (kWarps - 1)) start_word(a.counters + cta, a.call);
        word_started = true;
        // Q fragments, straight from global memory; rows past the unit's are zero
        WarpRows<D, MT> rw;
        rw.clear();
        int row_pos[MT][2];          // the rows' positions
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = mt * 16 + h * 8 + g;
                const bool live = r < rows;
                const int tok = live ? r / sq.group : 0, head = live ? r - tok * sq.group : 0;
                row_pos[mt][h] = cl.p0 + (live ? tok : cl.n - 1);
                const uint16_t *src = a.q + (size_t)(cl.t0 + tok) * a.q_stride + (size_t)(hk * sq.group + head) * D + 2 * t4;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    rw.q[mt][ks][h] = live ? *reinterpret_cast<const uint32_t *>(src + ks * 16) : 0u;
                    rw.q[mt][ks][2 + h] = live ? *reinterpret_cast<const uint32_t *>(src + ks * 16 + 8) : 0u;
                }
            }
        int stage = 0;
        for (; c < c_end; c += kWarps) {
            cp_async_wait<NS - 2>();
            __syncwarp();
            {
                const int id = next_id;
                next_id = page_of(c + NS * kWarps);
                load(c + (NS - 1) * kWarps, stage == 0 ? NS - 1 : stage - 1, id);
            }
            const uint32_t sk = ring + stage * L::kStage, sv = sk + L::kHalf;
            const int k0 = key_of(c);
            const bool whole = (k0 >= all_lo && k0 + kChunk <= all_hi) || k0 + kChunk <= all_shi;
            rw.chunk(sk, sv, a.scale_log2, whole, lane, [&](int mt, int h) {
                const RowKeys rk = paged_row(sq, row_pos[mt][h]);
                return seen_bits(rk.lo, rk.hi, rk.slo, rk.shi, k0);
            });
            __syncwarp();
            stage = stage + 1 == NS ? 0 : stage + 1;
        }
        cp_async_wait<0>();
        // ---- the four warps' rows become one
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                rw.l[mt][h] += __shfl_xor_sync(0xffffffffu, rw.l[mt][h], 1);
                rw.l[mt][h] += __shfl_xor_sync(0xffffffffu, rw.l[mt][h], 2);
                if (t4 == 0) {
                    s_m[warp][mt * 16 + h * 8 + g] = rw.m[mt][h];
                    s_l[warp][mt * 16 + h * 8 + g] = rw.l[mt][h];
                }
            }
        __syncthreads();     // every warp is past its ring too
        float *warp_o = reinterpret_cast<float *>(smem);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = mt * 16 + h * 8 + g;
                const float top = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
                const float f = rw.m[mt][h] > -INFINITY ? ex2(rw.m[mt][h] - top) : 0.f;
                float *dst = warp_o + ((size_t)warp * 16 * MT + r) * L::kRow + 2 * t4;
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *reinterpret_cast<float2 *>(dst + n * 8) = make_float2(rw.acc[mt][n][2 * h] * f, rw.acc[mt][n][2 * h + 1] * f);
            }
        __syncthreads();
        const bool begins = c_at == 0, ends = c_end == cl.count;
        if (flat && !(begins && ends)) {
            first_cta = (int)(unit_begin / per);
            last_cta = (int)((unit_end - 1) / per);
        }
        auto store = [&](int r, int col, const float (&x)[4], float inv) {
            const int tok = r / sq.group, head = hk * sq.group + r - tok * sq.group;
            const size_t at = ((size_t)(cl.t0 + tok) * sq.H + head) * D + col;
            if (a.o_bf16)
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.o) + at) =
                    make_uint2(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv));
            else
                *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + at) =
                    make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
        };
        auto store_lse = [&](int r, float top, float lsum) {
            const int tok = r / sq.group, head = hk * sq.group + r - tok * sq.group;
            if (a.lse)
                a.lse[(size_t)head * sq.T + cl.t0 + tok] = lsum > 0.f ? (top + lg2(lsum)) * 0.6931471805599453f : -INFINITY;
        };
        // NI four-column items of the pair's rows per thread, from item e0 on,
        // summed over the pieces; 16 / NI pieces at a time
        auto join = [&](auto ni, int e0) {
            constexpr int NI = decltype(ni)::value, B = 16 / NI;
            float x[NI][4] = {}, top[NI], lsum[NI] = {};
#pragma unroll
            for (int i = 0; i < NI; ++i) top[i] = -INFINITY;
            for (int p0 = first_cta; p0 <= last_cta; p0 += B) {
                float2 ml[B][NI];
                float4 f[B][NI];
#pragma unroll
                for (int j = 0; j < B; ++j)
#pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        const int e = e0 + threadIdx.x + i * 32 * kWarps, r = e / (D / 4), col = (e % (D / 4)) * 4;
                        const int p = p0 + j;
                        const size_t row = ((size_t)p * 2 + (p == first_cta ? 1 : 0)) * 16 * MT + r;
                        ml[j][i] = make_float2(-INFINITY, 0.f);
                        f[j][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (p <= last_cta && r < rows) {
                            ml[j][i] = __ldcg(reinterpret_cast<const float2 *>(a.part_ml + row * 2));
                            f[j][i] = __ldcg(reinterpret_cast<const float4 *>(a.part_o + row * D + col));
                        }
                    }
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    float t2 = top[i];
#pragma unroll
                    for (int j = 0; j < B; ++j) t2 = fmaxf(t2, ml[j][i].x);
                    if (!(t2 > -INFINITY)) continue;
                    const float old = ex2(top[i] - t2);
                    x[i][0] *= old, x[i][1] *= old, x[i][2] *= old, x[i][3] *= old;
                    lsum[i] *= old;
#pragma unroll
                    for (int j = 0; j < B; ++j) {
                        const float now = ex2(ml[j][i].x - t2);
                        x[i][0] += f[j][i].x * now;
                        x[i][1] += f[j][i].y * now;
                        x[i][2] += f[j][i].z * now;
                        x[i][3] += f[j][i].w * now;
                        lsum[i] += ml[j][i].y * now;
                    }
                    top[i] = t2;
                }
            }
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = e0 + threadIdx.x + i * 32 * kWarps, r = e / (D / 4), col = (e % (D / 4)) * 4;
                if (r >= rows) continue;
                store(r, col, x[i], lsum[i] > 0.f ? 1.f / lsum[i] : 0.f);
                if (col == 0) store_lse(r, top[i], lsum[i]);
            }
        };
        const size_t slot = (size_t)cta * 2 + (begins ? 1 : 0);
        for (int e = threadIdx.x; e < rows * (D / 4); e += blockDim.x) {
            const int r = e / (D / 4), col = (e % (D / 4)) * 4;
            float x[4] = {};
            float top = -INFINITY, lsum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 f = *reinterpret_cast<const float4 *>(warp_o + ((size_t)w * 16 * MT + r) * L::kRow + col);
                x[0] += f.x, x[1] += f.y, x[2] += f.z, x[3] += f.w;
                top = fmaxf(top, s_m[w][r]);
            }
#pragma unroll
            for (int w = 0; w < kWarps; ++w) lsum += s_m[w][r] > -INFINITY ? s_l[w][r] * ex2(s_m[w][r] - top) : 0.f;
            if constexpr (CLUSTER > 0) {
                // over the first warp's rows, which this thread alone has read here
                *reinterpret_cast<float4 *>(warp_o + (size_t)r * L::kRow + col) = make_float4(x[0], x[1], x[2], x[3]);
                if (col == 0) s_ml[r] = make_float2(top, lsum);
            } else if (begins && ends) {
                store(r, col, x, lsum > 0.f ? 1.f / lsum : 0.f);
                if (col == 0) store_lse(r, top, lsum);
            } else {
                *reinterpret_cast<float4 *>(a.part_o + (slot * 16 * MT + r) * D + col) = make_float4(x[0], x[1], x[2], x[3]);
                if (col == 0)
                    *reinterpret_cast<float2 *>(a.part_ml + (slot * 16 * MT + r) * 2) = make_float2(top, lsum);
            }
        }
        if constexpr (CLUSTER > 0) {
            cluster_sync();
            const int rank = cta % CLUSTER;
            for (int e = rank * 32 * kWarps + threadIdx.x; e < rows * (D / 4); e += CLUSTER * 32 * kWarps) {
                const int r = e / (D / 4), col = (e % (D / 4)) * 4;
                float2 ml[CLUSTER];
                float4 f[CLUSTER];
#pragma unroll
                for (int p = 0; p < CLUSTER; ++p) {
                    ml[p] = ld_cluster2(in_cluster(smem_u32(s_ml + r), p));
                    f[p] = ld_cluster4(in_cluster(smem_u32(warp_o + (size_t)r * L::kRow + col), p));
                }
                float x[4] = {}, top = -INFINITY, lsum = 0.f;
#pragma unroll
                for (int p = 0; p < CLUSTER; ++p) top = fmaxf(top, ml[p].x);
#pragma unroll
                for (int p = 0; p < CLUSTER; ++p) {
                    const float now = ml[p].x > -INFINITY ? ex2(ml[p].x - top) : 0.f;
                    x[0] += f[p].x * now;
                    x[1] += f[p].y * now;
                    x[2] += f[p].z * now;
                    x[3] += f[p].w * now;
                    lsum += ml[p].y * now;
                }
                store(r, col, x, lsum > 0.f ? 1.f / lsum : 0.f);
                if (col == 0) store_lse(r, top, lsum);
            }
            cluster_sync();      // the others have read this CTA's rows
            return;
        }
        if (!(begins && ends)) {
            // the head's last piece to arrive joins them, in order: the
            // barrier and the release order every thread's rows before the
            // count, the acquire the other pieces' rows after it
            __syncthreads();
            if (threadIdx.x == 0) {
                s_last = count_piece(a.counters + first_cta, a.call) == last_cta - first_cta;
                if (s_last) a.counters[first_cta] = a.call;
            }
            __syncthreads();
            if (s_last) {
                // 16 loads of each thread on their way at once
                const int items = rows * (D / 4);
                for (int e0 = 0; e0 < items; e0 += 4 * 32 * kWarps) {
                    const int left = (items - e0 + 32 * kWarps - 1) / (32 * kWarps);
                    if (left == 1) join(std::integral_constant<int, 1>(), e0);
                    else if (left == 2) join(std::integral_constant<int, 2>(), e0);
                    else join(std::integral_constant<int, 4>(), e0);
                }
            }
        }
        // ---- the next head, or the next sequence with new tokens
        pos = unit_begin + c_end;
        if (!flat || pos >= end) break;
        __syncthreads();     // the rows in shared memory have been read
        c_at = 0;
        if (++hk == sq.Hkv) {
            hk = 0;
            do cl = paged_chunks(sq, ++seq);
            while (cl.count == 0);
        }
    }
}

template <int D, int MT, int CLUSTER>
ra_status launch(const TokensLaunch &t, const TokensArgs &args, cudaStream_t stream) {
    auto kern = paged_tokens_kernel<D, MT, CLUSTER>;
    const int smem = (int)TokensSmem<D>::kBytes;
    static_assert(kWarps * 16 * MT * TokensSmem<D>::kRow * 4 <= TokensSmem<D>::kBytes, "the warps' rows fit in the rings");
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return set_error(RA_ERR_CUDA, "cudaFuncSetAttribute(MaxDynamicSharedMemorySize) failed");
    if constexpr (CLUSTER > 8)
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
            return set_error(RA_ERR_CUDA, "cudaFuncSetAttribute(NonPortableClusterSizeAllowed) failed");
    if constexpr (CLUSTER > 0)
        return launched(launch_dependent_clusters(kern, CLUSTER, (unsigned)t.ctas, 32 * kWarps, smem, stream, args));
    return launched(launch_dependent(kern, (unsigned)t.ctas, 32 * kWarps, smem, stream, args));
}

}  // namespace

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
    a.scale_log2 = t.scale_log2;
    a.status = t.status;
    static std::atomic<unsigned long long> calls{0};
    a.call = call_tag(calls.fetch_add(1, std::memory_order_relaxed));
    a.counters = t.counters;
    a.part_o = t.part_o;
    a.part_ml = t.part_ml;
    const int rows = t.seqs.max_new * t.seqs.group;
    auto go = [&](auto cluster) {
        constexpr int C = decltype(cluster)::value;
        if (t.d == 128) return rows <= 16 ? launch<128, 1, C>(t, a, stream) : launch<128, 2, C>(t, a, stream);
        return rows <= 16 ? launch<64, 1, C>(t, a, stream) : launch<64, 2, C>(t, a, stream);
    };
    if (t.cluster == 16) return go(std::integral_constant<int, 16>());
    if (t.cluster == 8) return go(std::integral_constant<int, 8>());
    if (t.cluster == 4) return go(std::integral_constant<int, 4>());
    if (t.cluster == 2) return go(std::integral_constant<int, 2>());
    return go(std::integral_constant<int, 0>());
}

}  // namespace ra
