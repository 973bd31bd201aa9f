// paged_rotary.cu -- appending new keys and values to a paged cache with the
// position rotation applied on the way, to the queries too.
//
// A token at position p turns the pair (x, y) number m of each head's first
// `rot` columns by the angle p f_m:
//   x' = x cos - y sin,  y' = x sin + y cos,
// the pair being columns m and m + rot / 2, or 2 m and 2 m + 1.  The angle is
// taken in turns modulo one (ra_rotary.cuh) and goes to sincospif.
//
// Bound by the bytes: each of q, k and v is read once and written once, 2 (H + 2
// H_kv) d 2 bytes a token.  The call is one list of items, each two 16-byte
// pieces of a head: the two that hold its pairs, or two to copy.  A block takes a
// run of the list, finds its tokens' places and computes their cosines once for
// all heads, while its first items are on their way.  One item of a thread at a time and five
// blocks to an SM: two at a time take the registers of one block, and were slower (20589
// tokens of 32 / 8 heads, d = 128: 84 us, 6.0 TB/s, against 90).
#include "paged_checks.h"
#include "ra_device.cuh"
#include "ra_launch.h"
#include "ra_paged.cuh"
#include "ra_rotary.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256, kTokens = 32;   // tokens a block meets at most
constexpr int kSeqs = kThreads - 1;      // sequences whose rows and lengths a block reads at once
constexpr int kSms = 152;
// cosines and sines of 8 pairs: 16 floats and 4 between them and the next, so
// that the 16-byte reads of 8 neighbouring threads meet in no bank
constexpr int kGroup = 20;

struct RotaryArgs {
    PagedSeqs seqs;
    const uint4 *q, *k, *v;
    uint4 *q_out, *k_pages, *v_pages;
    int64_t q_stride, out_stride, new_stride, page_stride;   // in 16-byte pieces
    const float *inv_freq;
    int H, Hkv, per_head;       // query heads (0: no queries), items of a head (d / 16)
    int turned;                 // items of a head that are turned (rot / 16)
    int pairs;                  // neighbouring columns are a pair
    int items, chunk;           // items of a token, of a block
    unsigned inverse;           // floor(2^32 / items): a division by items without one
    int shift, page_shift;      // log2 of per_head, of the page size
    unsigned *status;
};

__device__ __forceinline__ float2 bf16x2(uint32_t x) { return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)); }

__global__ void __launch_bounds__(kThreads, 5) paged_append_rotary_kernel(const RotaryArgs a) {
    const PagedSeqs &sq = a.seqs;
    __shared__ int64_t place[kTokens];       // a token's first piece in the pool, -1: not written
    __shared__ int position[kTokens];
    __shared__ int rows[kThreads], lens[kThreads];
    __shared__ unsigned live;                // tokens that belong to a sequence
    __shared__ unsigned long long fraction[64];
    __shared__ __align__(16) float turns[kTokens * 8 * kGroup];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    const int64_t total = (int64_t)sq.T * a.items;
    const int64_t first = (int64_t)blockIdx.x * a.chunk;
    const int64_t end = min(first + a.chunk, total);
    const int t0 = (int)(first / a.items);
    const int n_tok = (int)((end - 1) / a.items) - t0 + 1;

    struct Item {
        int tok, head, i;        // the token's number in the block; head: q's, k's, v's one after another
    };
    auto item_of = [&](int64_t e) {
        const unsigned in = (unsigned)(e - (int64_t)t0 * a.items);     // (a block's list is short)
        unsigned tok = __umulhi(in, a.inverse), r = in - tok * a.items;     // one too few at most
        if (r >= (unsigned)a.items) {
            r -= a.items;
            ++tok;
        }
        return Item{(int)tok, (int)(r >> a.shift), (int)(r & ((1u << a.shift) - 1))};
    };
    auto turned = [&](const Item &x) { return x.head < a.H + a.Hkv && x.i < a.turned; };
    // the item's first piece in its head, and from there to its second
    auto piece = [&](const Item &x) { return turned(x) && !a.pairs ? x.i : 2 * x.i; };
    auto second = [&](const Item &x) { return turned(x) && !a.pairs ? a.turned : 1; };
    uint4 x[2];
    auto load = [&](const Item &it) {
        const int64_t t = t0 + it.tok;
        const int in_head = piece(it);
        const uint4 *src = it.head < a.H ? a.q + t * a.q_stride + it.head * (2 * a.per_head)
                           : it.head < a.H + a.Hkv ? a.k + t * a.new_stride + (it.head - a.H) * (2 * a.per_head)
                                                   : a.v + t * a.new_stride + (it.head - a.H - a.Hkv) * (2 * a.per_head);
        x[0] = __ldcs(src + in_head);
        x[1] = __ldcs(src + in_head + second(it));
    };
    if (first + threadIdx.x < end) load(item_of(first + threadIdx.x));     // on its way while the places are found

    // ---- the tokens' places and positions, the frequencies
    // Few sequences: all their rows and lengths at once; many: by search.
    const bool few = sq.n_seqs <= kSeqs;
    if (few) {
        if ((int)threadIdx.x <= sq.n_seqs) rows[threadIdx.x] = paged_bound(sq, threadIdx.x);
        if ((int)threadIdx.x < sq.n_seqs) lens[threadIdx.x] = sq.seq_lens[threadIdx.x];
    }
    if (threadIdx.x >= kThreads - 64) {
        const int m = threadIdx.x - (kThreads - 64);
        if (m < a.turned * 8) fraction[m] = turn_fraction(a.inv_freq[m]);
    }
    if (few) __syncthreads();
    if (warp == 0) {
        const int t = t0 + lane;
        int s = 0, hi = sq.n_seqs;
        if (!few) {
            // the first token's sequence, 32 probes at a time, then for each lane's
            // token how many of the next 32 sequences begin at it or before
            while (hi - s > 1) {
                const int step = (hi - s + 31) / 32, at = s + lane * step;
                const bool below = at < hi && (lane == 0 || paged_bound(sq, at) <= t0);
                const int last = 31 - __clz(__ballot_sync(0xffffffffu, below));
                s += last * step;
                hi = min(hi, s + step);
            }
            const int lo = s, next = lo + 1 + lane < sq.n_seqs ? paged_bound(sq, lo + 1 + lane) : 0x7fffffff;
#pragma unroll
            for (int i = 0; i < 32; ++i) s += __shfl_sync(0xffffffffu, next, i) <= t ? 1 : 0;
            hi = s == lo + 32 ? sq.n_seqs : s;
        }
        while (hi - s > 1) {
            const int mid = (s + hi) >> 1;
            if ((few ? rows[mid] : paged_bound(sq, mid)) <= t) s = mid;
            else hi = mid;
        }
        const int c0 = few ? rows[s] : paged_bound(sq, s), c1 = few ? rows[s + 1] : paged_bound(sq, s + 1);
        bool in = lane < n_tok && t >= c0 && t < c1;
        int64_t dst = -1, p = 0;
        if (in) {
            const int i = t - c0;
            const int64_t before = (int64_t)(few ? lens[s] : sq.seq_lens[s]) - (c1 - c0), pos = before + i;
            p = pos;
            int id = -1;
            bool bad = false;
            const int64_t nth = pos >> a.page_shift;
            if (pos >= 0 && nth < sq.max_pages) id = sq.table[(size_t)s * sq.max_pages + nth];
            if (sq.parents) {
                if (i < kTreeMost) {
                    int depth = 0;
                    for (int j = tree_parent(sq.parents, c0, i, bad); j >= 0; j = tree_parent(sq.parents, c0, j, bad)) ++depth;
                    p = before + depth;
                } else {
                    in = false;
                }
            }
            if (in && id >= 0 && id < sq.n_pages)
                dst = (int64_t)id * a.page_stride + (pos & (sq.page - 1)) * (int64_t)(a.Hkv * 2 * a.per_head);
            else bad = true;
            if (bad) atomicOr(a.status, RA_DEV_PAGE_BIT);
        }
        place[lane] = dst;
        position[lane] = (int)p;
        const unsigned all = __ballot_sync(0xffffffffu, in);
        if (lane == 0) live = all;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < n_tok * a.turned * 8; e += kThreads) {
        const int tok = e / (a.turned * 8), m = e - tok * a.turned * 8;
        float s, c;
        sincospif(half_turns(position[tok], fraction[m]), &s, &c);
        float *to = turns + (tok * 8 + (m >> 3)) * kGroup + (m & 7);
        to[0] = c;
        to[8] = s;
    }
    __syncthreads();

    for (int64_t e = first + threadIdx.x; e < end; e += kThreads) {
        const Item it = item_of(e);
        if (e >= first + kThreads) load(it);
        if (!((live >> it.tok) & 1u)) continue;
        if (turned(it)) {
            const float4 *cs = reinterpret_cast<const float4 *>(turns + (it.tok * 8 + it.i) * kGroup);
            float c[8], s[8];
            *reinterpret_cast<float4 *>(c) = cs[0];
            *reinterpret_cast<float4 *>(c + 4) = cs[1];
            *reinterpret_cast<float4 *>(s) = cs[2];
            *reinterpret_cast<float4 *>(s + 4) = cs[3];
            uint32_t *w0 = reinterpret_cast<uint32_t *>(&x[0]), *w1 = reinterpret_cast<uint32_t *>(&x[1]);
            if (a.pairs) {
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    uint32_t &word = w < 4 ? w0[w] : w1[w - 4];
                    const float2 v = bf16x2(word);
                    word = pack_bf16x2(v.x * c[w] - v.y * s[w], v.x * s[w] + v.y * c[w]);
                }
            } else {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float2 u = bf16x2(w0[w]), v = bf16x2(w1[w]);
                    w0[w] = pack_bf16x2(u.x * c[2 * w] - v.x * s[2 * w], u.y * c[2 * w + 1] - v.y * s[2 * w + 1]);
                    w1[w] = pack_bf16x2(u.x * s[2 * w] + v.x * c[2 * w], u.y * s[2 * w + 1] + v.y * c[2 * w + 1]);
                }
            }
        }
        uint4 *dst;
        if (it.head < a.H) {
            dst = a.q_out + (int64_t)(t0 + it.tok) * a.out_stride + it.head * (2 * a.per_head);
        } else {
            if (place[it.tok] < 0) continue;
            const bool key = it.head < a.H + a.Hkv;
            dst = (key ? a.k_pages : a.v_pages) + place[it.tok] + (it.head - a.H - (key ? 0 : a.Hkv)) * (2 * a.per_head);
        }
        const int in_head = piece(it);
        dst[in_head] = x[0];
        dst[in_head + second(it)] = x[1];
    }
}

}  // namespace
}  // namespace ra

extern "C" ra_status ra_paged_append_rotary(const void *q, const void *k_new, const void *v_new, void *q_out, void *k_pages,
                                            void *v_pages, const int32_t *block_table, const int32_t *seq_lens,
                                            const int32_t *cu_new, const int32_t *parents, const float *inv_freq,
                                            int64_t T, int64_t n_seqs, int64_t H, int64_t H_kv, int d, int rot,
                                            int64_t n_pages, int64_t page_size, int64_t page_stride, int64_t max_pages,
                                            int64_t q_stride, int64_t q_out_stride, int64_t new_stride, unsigned flags,
                                            void *workspace, size_t workspace_bytes, void *stream) {
    using namespace ra;
    if (flags & ~RA_FLAG_ROTARY_PAIRS) return set_error(RA_ERR_INVALID_ARG, "unknown flag bits");
    ra_status st = check_heads(H_kv, H_kv, d);
    if (st != RA_OK) return st;
    if (H < 0) return set_error(RA_ERR_SHAPE, "sizes must be non-negative");
    if (H > (int64_t)1 << 16) return set_error(RA_ERR_UNSUPPORTED, "H beyond the supported range");
    if ((st = check_cache(T, n_seqs, H_kv, d, n_pages, page_size, page_stride, max_pages)) != RA_OK) return st;
    if (rot < 16 || rot > d || rot % 16)
        return set_error(RA_ERR_UNSUPPORTED, "the rotated columns must be a multiple of 16, at least 16 and at most d");
    const struct { int64_t stride, heads; } rows[] = {{new_stride, H_kv}, {q_stride, H}, {q_out_stride, H}};
    for (const auto &r : rows) {
        if (r.heads == 0) continue;
        if (r.stride < r.heads * d) return set_error(RA_ERR_SHAPE, "a token stride is smaller than its heads: tokens would overlap");
        if (r.stride % 8) return set_error(RA_ERR_ALIGNMENT, "token strides must be multiples of 8 elements (16 bytes)");
        if (r.stride >= kMostStride) return set_error(RA_ERR_UNSUPPORTED, "a token stride beyond the supported range");
    }
    if (T == 0 || n_seqs == 0) return RA_OK;
    if (n_pages == 0 || max_pages == 0) return set_error(RA_ERR_SHAPE, "new tokens need pages to lie in");
    if ((st = check_pointers({k_new, v_new, k_pages, v_pages, workspace}, {block_table, seq_lens, cu_new, inv_freq})) != RA_OK) return st;
    if (H > 0 && (st = check_pointers({q, q_out}, {})) != RA_OK) return st;
    if (H > 0 && q == q_out && q_stride != q_out_stride && T > 1)
        return set_error(RA_ERR_INVALID_ARG, "queries rotated in place keep their token stride");
    if (!aligned(parents, 4)) return set_error(RA_ERR_ALIGNMENT, "the int32 and fp32 vectors must be 4-byte aligned");
    if (H > 0) {
        // rotated queries go out while other blocks still read (q itself apart, which
        // each thread reads where it writes)
        const TokenRows from{q, q_stride, H * d}, to{q_out, q_out_stride, H * d};
        if ((q != q_out && rows_meet(from, to, T)) || rows_meet({k_new, new_stride, H_kv * d}, to, T) ||
            rows_meet({v_new, new_stride, H_kv * d}, to, T))
            return set_error(RA_ERR_INVALID_ARG, "q_out must overlap neither k_new nor v_new, nor q unless it is q");
    }
    if (workspace_bytes < RA_WORKSPACE_MIN_BYTES)
        return set_error(RA_ERR_INVALID_ARG, "workspace smaller than RA_WORKSPACE_MIN_BYTES");
    RotaryArgs a{};
    a.seqs.table = block_table;
    a.seqs.seq_lens = seq_lens;
    a.seqs.cu_q = cu_new;
    a.seqs.parents = parents;
    a.seqs.n_seqs = (int)n_seqs;
    a.seqs.T = (int)T;
    a.seqs.max_pages = (int)max_pages;
    a.seqs.page = (int)page_size;
    a.seqs.n_pages = (int)n_pages;
    a.q = static_cast<const uint4 *>(q);
    a.k = static_cast<const uint4 *>(k_new);
    a.v = static_cast<const uint4 *>(v_new);
    a.q_out = static_cast<uint4 *>(q_out);
    a.k_pages = static_cast<uint4 *>(k_pages);
    a.v_pages = static_cast<uint4 *>(v_pages);
    a.q_stride = q_stride / 8;
    a.out_stride = q_out_stride / 8;
    a.new_stride = new_stride / 8;
    a.page_stride = page_stride / 8;
    a.inv_freq = inv_freq;
    a.H = (int)H;
    a.Hkv = (int)H_kv;
    a.per_head = d / 16;
    a.turned = rot / 16;
    a.pairs = (flags & RA_FLAG_ROTARY_PAIRS) != 0;
    a.items = (int)((H + 2 * H_kv) * a.per_head);
    a.inverse = (unsigned)(((int64_t)1 << 32) / a.items);
    a.shift = d == 128 ? 3 : 2;
    while ((int64_t)1 << a.page_shift < page_size) ++a.page_shift;
    a.status = static_cast<unsigned *>(workspace);
    // an item to a thread while that fills the SMs, then several, of no more tokens than a block holds
    const int64_t total = T * a.items;
    int64_t chunk = kThreads;
    while (chunk < 8 * kThreads && total / chunk > 8 * kSms) chunk *= 2;
    if (chunk > (int64_t)(kTokens - 1) * a.items) chunk = (int64_t)(kTokens - 1) * a.items;
    a.chunk = (int)chunk;
    const int64_t blocks = (total + chunk - 1) / chunk;
    if (blocks > 0x7fffffffLL) return set_error(RA_ERR_UNSUPPORTED, "too many blocks for one launch");
    return launched(launch_dependent(paged_append_rotary_kernel, (unsigned)blocks, kThreads, 0, static_cast<cudaStream_t>(stream), a));
}
