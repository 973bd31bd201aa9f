// attn_paged.cu -- attention of new tokens over a paged key/value cache: the
// entry points, their checks and launches, the join of split keys, and the
// copy of new keys and values into the cache.
//
// ra_paged_attn_fwd runs the tensor-core forward (attn_fwd_kernel.cuh,
// KEYS_PAGED): units of up to 256 rows (the query heads of one key/value head
// by consecutive new tokens), key tiles of 128 gathered page by page with TMA.
// Where there are few units, each unit's key tiles are cut into parts that run
// as CTAs of their own and are joined by their LSE.  Bound by the tensor cores'
// pace (about 1.35 us for 128 keys by 256 rows at d = 128) and a CTA's fixed 8
// us: 512 tokens over 32768 keys, 32 / 8 heads, 202 us in pages of 16 and 190 in
// pages of 128 (1350 and 1440 TFLOP/s); two prompts of 2048 tokens over 8192: 335
// us (1440 TFLOP/s), each call on other inputs (the same again: 190 us in pages of
// 16).  Few rows and few keys have forms of their own.
#include <cmath>

#include "attn_fwd_kernel.cuh"
#include "paged_launch.h"
#include "ra_launch.h"
#include "ra_tensor_map.h"

namespace ra {
namespace {

constexpr size_t kHeader = RA_WORKSPACE_MIN_BYTES;
constexpr int kSms = 152;               // GB300; only the choice of a split depends on it
constexpr size_t kPartBytes = (64u << 20) - (16u << 10);   // most bytes of a call's parts
constexpr size_t kCounters = kHeader, kCounterBytes = 4096;   // the few-row kernel's
static_assert(kPagedTokensCtas * 8 <= kCounterBytes, "one counter per CTA");

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }
bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// ------------------------------------------------------------------ join
// O = sum_i w_i O_i, w_i = exp(LSE_i - LSE), over a row's parts in order, so
// that the result does not depend on timing; rows of one part were written by
// the forward itself.  D / 4 lanes per row, 8 parts on their way at once:
// bound by the parts' bytes, most of which are still in L2.
struct JoinArgs {
    PagedSeqs seqs;
    const float *part_o, *part_lse;
    void *o;
    float *lse;
    int o_bf16;
};

template <int D>
__global__ void __launch_bounds__(256) paged_join_kernel(const JoinArgs a) {
    const PagedSeqs &q = a.seqs;
    constexpr int LANES = D / 4, AHEAD = 8;
    pdl_wait();
    const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LANES;
    const int col = threadIdx.x % LANES * 4;
    if (row >= (int64_t)q.T * q.H) return;
    const int tok = (int)(row / q.H), head = (int)(row - (int64_t)tok * q.H);
    // the last sequence starting at or before the token
    int lo = 0, hi = q.n_seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (paged_bound(q, mid) <= tok) lo = mid;
        else hi = mid;
    }
    const int i = tok - paged_bound(q, lo);
    if (i < 0 || i >= q.max_new || tok >= paged_bound(q, lo + 1)) return;    // behind the last sequence
    const int local = i / q.unit_tokens;
    const PagedUnit u = paged_unit(q, lo, local);
    const int parts = paged_split_count(q, paged_walk(q, u).end);
    if (parts == 1) return;
    const size_t rows = paged_unit_rows(q);
    const size_t unit = (size_t)paged_first_unit(q, lo) + local;
    const size_t first = ((unit * q.Hkv + head / q.group) * q.num_splits) * rows +
                         (size_t)(i - u.first) * q.group + head % q.group;
    float x[4] = {}, top = -INFINITY, sum = 0.f;
    for (int p0 = 0; p0 < parts; p0 += AHEAD) {
        float l[AHEAD];
        float4 f[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const size_t at = first + min(p0 + j, parts - 1) * rows;
            l[j] = a.part_lse[at];
            f[j] = *reinterpret_cast<const float4 *>(a.part_o + at * D + col);
        }
        float t2 = top;
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) t2 = fmaxf(t2, l[j]);
        if (!(t2 > -INFINITY)) continue;
        const float old = ex2((top - t2) * 1.4426950408889634f);
        x[0] *= old, x[1] *= old, x[2] *= old, x[3] *= old;
        sum *= old;
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            if (p0 + j >= parts) break;
            const float w = ex2((l[j] - t2) * 1.4426950408889634f);
            x[0] += f[j].x * w;
            x[1] += f[j].y * w;
            x[2] += f[j].z * w;
            x[3] += f[j].w * w;
            sum += w;
        }
        top = t2;
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    if (a.o_bf16)
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.o) + row * D + col) =
            make_uint2(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv));
    else
        *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + row * D + col) =
            make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    if (col == 0 && a.lse)
        a.lse[(size_t)head * q.T + tok] = sum > 0.f ? top + lg2(sum) * 0.6931471805599453f : -INFINITY;
}

// ------------------------------------------------------------------ plan
struct Paged {
    int64_t T, n_seqs, H, H_kv, n_pages, page, page_stride, max_pages, q_stride, max_new, max_len, window, sinks;
    int d;
    float scale;
};

// How a call is cut: tokens per unit, the most parts per unit, the parts' bytes.
struct Plan {
    int tile_tokens, splits, tail_share;    // the tensor-core form
    int64_t units;
    bool tokens, whole_pairs;   // the few-row form, with this many CTAs, in clusters or not
    int ctas, cluster;
    bool few;                   // the few-key form: units of its own, the keys it expects
    int64_t few_units, few_keys;
    size_t part_o, part_lse, total;
};

// The few-key form runs where a block of 64 rows sees few keys.  Chunks of 33 to
// L new tokens over L keys, few-key against tensor-core form in us: 40 sequences,
// 8 / 8 heads, d = 64: L = 40: 7.2 / 17.5, 100: 13.7 / 17.8, 160: 18.7 / 22.7,
// 250: 33 / 23; 32 / 8 heads: 14 / 20, 25 / 25, 41 / 37; d = 128, 8 / 8 heads:
// 12 / 21, 19 / 21, 43 / 27; 8 sequences, 16 / 8 heads: 6.0 / 7.8, 10.1 / 8.6.
bool few_keys(int64_t keys, int d) { return keys <= (d == 64 ? 128 : 64); }

Plan plan(Paged a) {
    // hints of any size: with the sizes that the checks admit nothing below leaves
    // 64 bits (pairs reach 2^40, keys 2^30, a part's bytes 2^58, of which 64 are tried)
    const int64_t cap = (int64_t)1 << 29;
    if (a.max_new > a.T) a.max_new = a.T;
    if (a.max_len > cap) a.max_len = cap;
    if (a.window > cap) a.window = cap;
    if (a.sinks > cap) a.sinks = cap;
    Plan p{};
    const int64_t group = a.H / a.H_kv;
    const int64_t active0 = a.n_seqs < a.T ? a.n_seqs : a.T;
    p.part_o = kCounters + kCounterBytes;
    // Few rows per key/value head: bound by the cache's bytes (see attn_paged_tokens.cu)
    if (a.max_new * group <= kPagedTokensRows) {
        p.tokens = true;
        int64_t seen = a.max_len;
        if (a.window > 0 && a.window + a.max_new + a.sinks < seen) seen = a.window + a.max_new + a.sinks;
        p.ctas = paged_tokens_ctas(active0 * a.H_kv, seen, a.n_seqs);
        p.whole_pairs = paged_tokens_whole(active0 * a.H_kv, seen, a.n_seqs);
        p.cluster = paged_tokens_cluster(active0 * a.H_kv, seen);
        const size_t rows = p.whole_pairs || p.cluster ? 0 : (size_t)2 * p.ctas * (a.max_new * group <= 16 ? 16 : 32);
        p.part_lse = p.part_o + round256(rows * a.d * 4);
        p.total = p.part_lse + round256(rows * 8);
        return p;
    }
    if (group <= kPagedFewRows) {
        const int unit = (int)(kPagedFewRows / group);
        p.few_units = paged_units(a.T, a.n_seqs, unit);
        p.few_keys = a.max_len;
        if (a.window > 0 && a.window + unit + a.sinks < p.few_keys) p.few_keys = a.window + unit + a.sinks;
        p.few = few_keys(p.few_keys, a.d);
        if (p.few) {
            p.total = p.part_o;
            return p;
        }
    }
    p.tile_tokens = (int)(128 / group);
    const int unit = 2 * p.tile_tokens;
    p.units = paged_units(a.T, a.n_seqs, unit);
    const int64_t rows = (a.max_new < unit ? a.max_new : unit) * group;
    const size_t part = (size_t)p.units * a.H_kv * rows * (a.d + 1) * 4;     // one part of every unit
    // The time of s parts, in us: a CTA costs about 8 and 1.35 a key tile (1.0 at
    // d = 64).  While one wave holds them all it is the longest CTA's; past that
    // the SMs' even share and a part of a CTA more, a smaller one where longer
    // sequences go first.  max_len bounds the lengths: several sequences are taken
    // to have half of it on average.  The parts are written and read at about 3 TB/s.
    //   512 tokens over 32768 keys, 32 / 8 heads, d = 128, s = 1, 2, 3, 4, 7:
    //   357, 199, 260, 210, 202; 8 ragged sequences of up to 700 tokens over 9000
    //   keys, 16 / 4 heads, d = 64, s = 1, 2, 3: 83, 116, 124 (s = 1 in the order of
    //   the sequences: 105); 4 of 300-500 over up to 16000, 32 / 8 heads, d = 128: 168,
    //   206, 222; 16 of 50-100 over up to 8000, 8 / 2 heads: 80, 55, 44, and 4: 50.
    const int64_t full = (a.T + unit - 1) / unit;
    const int64_t ctas = (full > active0 ? full : active0) * a.H_kv;
    int64_t keys = a.max_len;
    if (a.window > 0 && a.window + a.max_new + a.sinks < keys) keys = a.window + (a.max_new < unit ? a.max_new : unit) + a.sinks;
    const int64_t tiles = (keys + 127) / 128 + 1;
    const double tile = a.d == 128 ? 1.35 : 1.0, fixed = 8.0;
    const double mean = active0 > 1 && !(a.window > 0) ? 0.55 * (double)tiles : (double)tiles;
    const double late = a.n_seqs > 1 && a.n_seqs <= 32 ? 0.2 : 0.5;
    auto join = [&](int s) { return s > 1 ? 4.0 + (double)(a.T * a.H) * s * a.d * 8 / 3e6 : 0.0; };
    p.splits = 1;
    double best = 0;
    for (int s = 1; s <= 64 && (s == 1 || (tiles / s >= kSplitTiles && part * s <= kPartBytes)); ++s) {
        const double longest = fixed + tile * (double)((tiles + s - 1) / s);
        const double share = (double)ctas * (s * fixed + mean * tile) / kSms;
        const double t = (ctas * s <= kSms || longest > share + late * longest ? longest : share + late * longest) + join(s);
        if (s == 1 || t < best) {
            best = t;
            p.splits = s;
        }
    }
    // One sequence whose parts leave SMs idle: s long parts of each unit on SMs of
    // their own and a short last part, `rounds` of which follow one another on the
    // others and end with the long ones.  512 tokens over 32768 keys, 32 / 8 heads,
    // two parts against two and a short one: 219 / 197 us in pages of 16, 202 / 184
    // in pages of 128; 256 tokens 110 / 102.  Where the estimate promises less than
    // 5 % it does not hold: 1000 tokens over 16000 keys 171 / 183.
    for (int s = 1; active0 == 1 && s < 64 && s * ctas < kSms && part * (s + 1) <= kPartBytes; ++s) {
        const int64_t idle = kSms - s * ctas, rounds = (ctas + idle - 1) / idle;
        const double tail = ((double)tiles * tile / s - fixed * (double)(rounds - 1)) / (tile * ((double)rounds + 1.0 / s));
        const double longest = ((double)tiles - tail) / s;
        if (tail < kSplitTiles || longest < tail) continue;
        const double t = fixed + tile * longest + join(s + 1);
        if (t < 0.95 * best) {
            best = t;
            p.splits = s + 1;
            p.tail_share = (int)(1024.0 * tail / (double)tiles);
        }
    }
    p.part_lse = p.total = p.part_o;
    if (p.splits > 1) {
        p.part_lse = p.part_o + round256((size_t)p.units * a.H_kv * p.splits * rows * a.d * 4);
        p.total = p.part_lse + round256((size_t)p.units * a.H_kv * p.splits * rows * 4);
    }
    return p;
}

constexpr int64_t kMostStride = (int64_t)1 << 39;     // elements; a tensor map's strides stay below 2^40 bytes

ra_status check_heads(int64_t H, int64_t H_kv, int d) {
    if (d != 64 && d != 128) return set_error(RA_ERR_UNSUPPORTED, "head dimension d must be 64 or 128");
    if (H_kv < 1 || H_kv > H || H % H_kv)
        return set_error(RA_ERR_SHAPE, "the key/value head count must divide the query head count");
    if (H / H_kv > 128) return set_error(RA_ERR_UNSUPPORTED, "at most 128 query heads per key/value head");
    if (H > (int64_t)1 << 16) return set_error(RA_ERR_UNSUPPORTED, "H beyond the supported range");
    return RA_OK;
}

ra_status check_cache(int64_t T, int64_t n_seqs, int64_t H_kv, int d, int64_t n_pages, int64_t page,
                      int64_t page_stride, int64_t max_pages) {
    if (T < 0 || n_seqs < 0 || n_pages < 0 || max_pages < 0) return set_error(RA_ERR_SHAPE, "sizes must be non-negative");
    if (page < 16 || page > 65536 || (page & (page - 1)))
        return set_error(RA_ERR_UNSUPPORTED, "page_size must be a power of two, at least 16 and at most 65536");
    if (T > (int64_t)1 << 24 || n_seqs > (int64_t)1 << 24 || n_pages > (int64_t)1 << 30)
        return set_error(RA_ERR_UNSUPPORTED, "tokens, sequences or pages beyond the supported range");
    if (max_pages > ((int64_t)1 << 29) / page)
        return set_error(RA_ERR_UNSUPPORTED, "max_pages * page_size beyond the supported range (2^29 tokens)");
    if (page_stride < page * H_kv * d) return set_error(RA_ERR_SHAPE, "page_stride is smaller than a page: pages would overlap");
    if (page_stride % 8) return set_error(RA_ERR_ALIGNMENT, "page_stride must be a multiple of 8 elements (16 bytes)");
    if (page_stride >= kMostStride) return set_error(RA_ERR_UNSUPPORTED, "page_stride beyond the supported range");
    return RA_OK;
}

ra_status check(const Paged &a) {
    ra_status st = check_heads(a.H, a.H_kv, a.d);
    if (st != RA_OK) return st;
    if ((st = check_cache(a.T, a.n_seqs, a.H_kv, a.d, a.n_pages, a.page, a.page_stride, a.max_pages)) != RA_OK) return st;
    if (std::isnan(a.scale) || std::isinf(a.scale)) return set_error(RA_ERR_INVALID_ARG, "scale must be finite");
    if (a.q_stride < a.H * a.d) return set_error(RA_ERR_SHAPE, "q_stride is smaller than H * d: tokens would overlap");
    if (a.q_stride % 8) return set_error(RA_ERR_ALIGNMENT, "q_stride must be a multiple of 8 elements (16 bytes)");
    if (a.q_stride >= kMostStride) return set_error(RA_ERR_UNSUPPORTED, "q_stride beyond the supported range");
    if (a.max_new < 0 || a.max_len < 0) return set_error(RA_ERR_SHAPE, "max_new and max_len must be non-negative");
    if (a.window < 0) return set_error(RA_ERR_INVALID_ARG, "window must not be negative (0: none)");
    if (a.sinks < 0) return set_error(RA_ERR_INVALID_ARG, "sinks must not be negative");
    return RA_OK;
}

// ------------------------------------------------------------------ launch
// Pages of [page, H_kv, d], in boxes of `box` tokens of one head (KvTile).
// d = 64: {columns, tokens, pages}.  d = 128: {64 columns, 8 tokens, halves of
// all heads, groups of 8 tokens, pages}, a box holding both halves.
bool page_map(CUtensorMap *map, const void *base, const Paged &a, int box) {
    EncodeTiledFn enc = get_encode_fn();
    if (!enc) return false;
    const cuuint64_t token = (cuuint64_t)(a.H_kv * a.d * 2), page = (cuuint64_t)(a.page_stride * 2);
    const cuuint64_t dims3[3] = {(cuuint64_t)(a.H_kv * a.d), (cuuint64_t)a.page, (cuuint64_t)a.n_pages};
    const cuuint64_t strides3[2] = {token, page};
    const cuuint32_t box3[3] = {64, (cuuint32_t)box, 1};
    const cuuint64_t dims5[5] = {64, 8, (cuuint64_t)(2 * a.H_kv), (cuuint64_t)(a.page / 8), (cuuint64_t)a.n_pages};
    const cuuint64_t strides5[4] = {token, 128, 8 * token, page};
    const cuuint32_t box5[5] = {64, 8, 2, (cuuint32_t)(box / 8), 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    const bool halves = a.d == 128;
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, halves ? 5 : 3, const_cast<void *>(base), halves ? dims5 : dims3,
               halves ? strides5 : strides3, halves ? box5 : box3, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [T, H, d] with a token stride, in boxes of 64 columns by a group's heads by tile_tokens tokens
bool query_map(CUtensorMap *map, const void *base, const Paged &a, int tile_tokens) {
    EncodeTiledFn enc = get_encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)a.d, (cuuint64_t)a.H, (cuuint64_t)a.T};
    cuuint64_t strides[2] = {(cuuint64_t)(a.d * 2), (cuuint64_t)(a.q_stride * 2)};
    cuuint32_t bx[3] = {64, (cuuint32_t)(a.H / a.H_kv), (cuuint32_t)tile_tokens}, estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, bx, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

PagedSeqs sequences(const Paged &a, const int *table, const int *seq_lens, const int *cu_q) {
    PagedSeqs s{};
    s.table = table;
    s.seq_lens = seq_lens;
    s.cu_q = cu_q;
    s.n_seqs = (int)a.n_seqs;
    s.T = (int)a.T;
    s.max_pages = (int)a.max_pages;
    s.page = (int)a.page;
    s.n_pages = (int)a.n_pages;
    s.H = (int)a.H;
    s.Hkv = (int)a.H_kv;
    s.group = (int)(a.H / a.H_kv);
    s.max_new = (int)(a.max_new < a.T ? a.max_new : a.T);
    const int64_t cap = (int64_t)1 << 29;      // at least as long as any cache
    s.window = (int)(a.window < cap ? a.window : cap);
    s.sinks = (int)(a.sinks < cap ? a.sinks : cap);
    return s;
}

template <int D, bool F32>
ra_status launch_chunks(const Paged &a, const Plan &p, const AttnArgs &args, const void *q, const void *k,
                        const void *v, cudaStream_t stream) {
    CUtensorMap mq, mk, mv;
    if (!query_map(&mq, q, a, p.tile_tokens) || !page_map(&mk, k, a, args.page_box) || !page_map(&mv, v, a, args.page_box))
        return set_error(RA_ERR_CUDA, "cuTensorMapEncodeTiled failed for the q and page maps");
    auto kern = attn_fwd_kernel<D, F32, false, KEYS_PAGED>;
    const int smem = (int)AttnSmem<D>::kBytes;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return set_error(RA_ERR_CUDA, "cudaFuncSetAttribute(MaxDynamicSharedMemorySize) failed");
    const int64_t grid = p.units * a.H_kv * p.splits;
    if (grid > 0x7fffffffLL) return set_error(RA_ERR_UNSUPPORTED, "too many query tiles for one launch");
    return launched(launch_dependent(kern, (unsigned)grid, 384, smem, stream, mq, mk, mv, mq, args));
}

template <int D>
ra_status launch_paged(const Paged &a, const int *table, const int *seq_lens, const int *cu_q, const void *q,
                       const void *k, const void *v, void *o, float *lse, bool o_bf16, uint8_t *workspace,
                       cudaStream_t stream) {
    const Plan p = plan(a);
    const float scale_log2 = (a.scale > 0.f ? a.scale : 1.0f / std::sqrt((float)a.d)) * 1.4426950408889634f;
    if (p.tokens) {
        TokensLaunch t{};
        t.seqs = sequences(a, table, seq_lens, cu_q);
        t.seqs.unit_tokens = t.seqs.max_new;        // a sequence's tokens are one unit
        t.q = q;
        t.k = k;
        t.v = v;
        t.q_stride = a.q_stride;
        t.page_stride = a.page_stride;
        t.o = o;
        t.lse = lse;
        t.o_bf16 = o_bf16;
        t.d = D;
        t.whole_pairs = p.whole_pairs;
        t.cluster = p.cluster;
        t.ctas = p.ctas;
        t.scale_log2 = scale_log2;
        t.status = reinterpret_cast<unsigned *>(workspace);
        t.counters = reinterpret_cast<unsigned long long *>(workspace + kCounters);
        t.part_o = reinterpret_cast<float *>(workspace + p.part_o);
        t.part_ml = reinterpret_cast<float *>(workspace + p.part_lse);
        return launch_paged_tokens(t, stream);
    }
    if (p.few) {
        PagedFewLaunch t{};
        t.seqs = sequences(a, table, seq_lens, cu_q);
        t.seqs.unit_tokens = kPagedFewRows / t.seqs.group;
        t.q = q;
        t.k = k;
        t.v = v;
        t.q_stride = a.q_stride;
        t.page_stride = a.page_stride;
        t.o = o;
        t.lse = lse;
        t.o_bf16 = o_bf16;
        t.d = D;
        t.units = (int)p.few_units;
        t.keys = p.few_keys;
        t.scale_log2 = scale_log2;
        t.status = reinterpret_cast<unsigned *>(workspace);
        return launch_paged_few(t, stream);
    }
    AttnArgs args{};
    args.o = o;
    args.lse = lse;
    args.status = reinterpret_cast<unsigned *>(workspace);
    args.B = args.H = args.N = 1;
    args.layout = RA_CONTIGUOUS;
    args.causal = 1;
    args.scale_log2 = scale_log2;
    args.num_q_ranks = 1;
    args.q_rank_fixed = args.kv_rank_fixed = -1;
    args.num_steps = 1;
    args.kv_group = 1;
    args.seqs = sequences(a, table, seq_lens, cu_q);
    args.seqs.unit_tokens = 2 * p.tile_tokens;
    args.seqs.num_splits = p.splits;
    args.seqs.tail_share = p.tail_share;
    args.n_units = (int)p.units;
    args.tile_tokens = p.tile_tokens;
    args.page_box = (int)(a.page < 128 ? a.page : 128);
    args.o_bf16 = o_bf16 ? 1 : 0;
    args.part_o = reinterpret_cast<float *>(workspace + p.part_o);
    args.part_lse = reinterpret_cast<float *>(workspace + p.part_lse);
    const bool f32 = p.splits > 1 || !o_bf16;
    if (p.splits > 1 && a.T * a.H > (int64_t)1 << 31) return set_error(RA_ERR_UNSUPPORTED, "too many rows for one launch");
    const ra_status st = f32 ? launch_chunks<D, true>(a, p, args, q, k, v, stream)
                             : launch_chunks<D, false>(a, p, args, q, k, v, stream);
    if (st != RA_OK || p.splits == 1) return st;
    JoinArgs j{args.seqs, args.part_o, args.part_lse, o, lse, o_bf16 ? 1 : 0};
    const int64_t per_block = 256 / (D / 4), blocks = (a.T * a.H + per_block - 1) / per_block;
    return launched(launch_dependent(paged_join_kernel<D>, (unsigned)blocks, 256, 0, stream, j));
}

// ------------------------------------------------------------------ append
// Row i of sequence s's n new rows goes to position seq_lens[s] - n + i.  A
// token's bytes are one run on both sides; a block copies up to kAppendTokens
// tokens, each thread four 16-byte pieces of keys and of values at a time.
// Bound by HBM: 4 * H_kv * d * 2 bytes per token; 20589 tokens of 8 heads, d =
// 128: 29 us, 5.8 TB/s; 64 tokens 2.7 us, the launch.
struct AppendArgs {
    PagedSeqs seqs;
    const uint4 *k_new, *v_new;
    uint4 *k_pages, *v_pages;
    int64_t new_stride, page_stride;   // in 16-byte pieces
    int pieces, tokens;                // pieces of a token, tokens of a block
    unsigned *status;
};

constexpr int kAppendThreads = 256, kAppendTokens = 32;

__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const AppendArgs a) {
    const PagedSeqs &q = a.seqs;
    __shared__ int64_t dst_of[kAppendTokens];
    pdl_wait();
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
    const int n_tok = (int)min((int64_t)a.tokens, q.T - t0);
    if ((int)threadIdx.x < n_tok) {
        const int64_t t = t0 + threadIdx.x;
        int64_t dst = -1;
        int lo = 0, hi = q.n_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (paged_bound(q, mid) <= t) lo = mid;
            else hi = mid;
        }
        const int c0 = paged_bound(q, lo), c1 = paged_bound(q, lo + 1);
        if (t >= c0 && t < c1) {
            const int64_t pos = (int64_t)q.seq_lens[lo] - (c1 - t);
            int id = -1;
            if (pos >= 0 && pos / q.page < q.max_pages) id = q.table[(size_t)lo * q.max_pages + pos / q.page];
            if (id >= 0 && id < q.n_pages) dst = (int64_t)id * a.page_stride + (pos & (q.page - 1)) * a.pieces;
            else atomicOr(a.status, RA_DEV_PAGE_BIT);
        }
        dst_of[threadIdx.x] = dst;
    }
    __syncthreads();
    constexpr int U = 4;
    const int total = n_tok * a.pieces;
    for (int e0 = threadIdx.x; e0 < total; e0 += U * kAppendThreads) {
        uint4 k[U], v[U];
        int64_t dst[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int e = e0 + j * kAppendThreads;
            dst[j] = -1;
            if (e >= total) continue;
            const int i = e / a.pieces, c = e - i * a.pieces;
            if (dst_of[i] < 0) continue;
            dst[j] = dst_of[i] + c;
            const int64_t src = (t0 + i) * a.new_stride + c;
            k[j] = __ldcs(a.k_new + src);
            v[j] = __ldcs(a.v_new + src);
        }
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (dst[j] >= 0) {
                a.k_pages[dst[j]] = k[j];
                a.v_pages[dst[j]] = v[j];
            }
    }
}

}  // namespace
}  // namespace ra

extern "C" {

size_t ra_paged_attn_workspace_bytes(int64_t T, int64_t n_seqs, int64_t H, int64_t H_kv, int d, int64_t max_new,
                                     int64_t max_len, int64_t window, int64_t sinks) {
    if (T < 0 || n_seqs < 0 || max_new < 0 || max_len < 0 || window < 0 || sinks < 0 || H_kv < 1 || H < H_kv ||
        H % H_kv || H / H_kv > 128 || H > (int64_t)1 << 16 || (d != 64 && d != 128) || T > (int64_t)1 << 24 ||
        n_seqs > (int64_t)1 << 24)
        return 0;
    ra::Paged a{};
    a.T = T, a.n_seqs = n_seqs, a.H = H, a.H_kv = H_kv, a.d = d, a.max_new = max_new, a.max_len = max_len;
    a.window = window, a.sinks = sinks;
    return ra::plan(a).total;
}

ra_status ra_paged_attn_fwd(const void *q, const void *k_pages, const void *v_pages, const int32_t *block_table,
                            const int32_t *seq_lens, const int32_t *cu_q, void *o, float *lse, int64_t T,
                            int64_t n_seqs, int64_t H, int64_t H_kv, int d, int64_t n_pages, int64_t page_size,
                            int64_t page_stride, int64_t max_pages, int64_t q_stride, int64_t max_new,
                            int64_t max_len, int64_t window, int64_t sinks, float scale, unsigned flags,
                            void *workspace, size_t workspace_bytes, void *stream) {
    using namespace ra;
    if (flags & ~RA_FLAG_O_BF16) return set_error(RA_ERR_INVALID_ARG, "unknown flag bits");
    Paged a{T, n_seqs, H, H_kv, n_pages, page_size, page_stride, max_pages, q_stride, max_new, max_len, window, sinks,
            d, scale};
    const ra_status st = check(a);
    if (st != RA_OK) return st;
    if (T == 0 || n_seqs == 0 || max_new == 0) return RA_OK;
    if (n_pages == 0 || max_pages == 0) return set_error(RA_ERR_SHAPE, "new tokens need pages to lie in");
    const void *ptrs[] = {q, k_pages, v_pages, o, workspace};
    for (const void *p : ptrs) {
        if (!p) return set_error(RA_ERR_INVALID_ARG, "null pointer argument");
        if (!aligned(p, 16)) return set_error(RA_ERR_ALIGNMENT, "every tensor pointer must be 16-byte aligned");
    }
    const void *ints[] = {block_table, seq_lens, cu_q};
    for (const void *p : ints) {
        if (!p) return set_error(RA_ERR_INVALID_ARG, "null pointer argument");
        if (!aligned(p, 4)) return set_error(RA_ERR_ALIGNMENT, "block_table, seq_lens and cu_q must be 4-byte aligned");
    }
    if (!aligned(lse, 4)) return set_error(RA_ERR_ALIGNMENT, "lse must be 4-byte aligned");
    // a CTA of the few-row form counts its 16-key chunks in 31 bits
    const int64_t active = n_seqs < T ? n_seqs : T;
    if ((double)(active * H_kv) * (double)(max_pages * page_size) > 0x1p43)
        return set_error(RA_ERR_UNSUPPORTED, "sequences * H_kv * max_pages * page_size beyond the supported range (2^43)");
    if (workspace_bytes < plan(a).total)
        return set_error(RA_ERR_INVALID_ARG, "workspace smaller than ra_paged_attn_workspace_bytes()");
    auto launch = d == 128 ? launch_paged<128> : launch_paged<64>;
    return launch(a, block_table, seq_lens, cu_q, q, k_pages, v_pages, o, lse, (flags & RA_FLAG_O_BF16) != 0,
                  static_cast<uint8_t *>(workspace), static_cast<cudaStream_t>(stream));
}

ra_status ra_paged_append(const void *k_new, const void *v_new, void *k_pages, void *v_pages,
                          const int32_t *block_table, const int32_t *seq_lens, const int32_t *cu_new, int64_t T,
                          int64_t n_seqs, int64_t H_kv, int d, int64_t n_pages, int64_t page_size,
                          int64_t page_stride, int64_t max_pages, int64_t new_stride, void *workspace,
                          size_t workspace_bytes, void *stream) {
    using namespace ra;
    ra_status st = check_heads(H_kv, H_kv, d);
    if (st != RA_OK) return st;
    if ((st = check_cache(T, n_seqs, H_kv, d, n_pages, page_size, page_stride, max_pages)) != RA_OK) return st;
    if (new_stride < H_kv * d) return set_error(RA_ERR_SHAPE, "new_stride is smaller than H_kv * d: tokens would overlap");
    if (new_stride % 8) return set_error(RA_ERR_ALIGNMENT, "new_stride must be a multiple of 8 elements (16 bytes)");
    if (new_stride >= kMostStride) return set_error(RA_ERR_UNSUPPORTED, "new_stride beyond the supported range");
    if (T == 0 || n_seqs == 0) return RA_OK;
    if (n_pages == 0 || max_pages == 0) return set_error(RA_ERR_SHAPE, "new tokens need pages to lie in");
    const void *ptrs[] = {k_new, v_new, k_pages, v_pages, workspace};
    for (const void *p : ptrs) {
        if (!p) return set_error(RA_ERR_INVALID_ARG, "null pointer argument");
        if (!aligned(p, 16)) return set_error(RA_ERR_ALIGNMENT, "every tensor pointer must be 16-byte aligned");
    }
    const void *ints[] = {block_table, seq_lens, cu_new};
    for (const void *p : ints) {
        if (!p) return set_error(RA_ERR_INVALID_ARG, "null pointer argument");
        if (!aligned(p, 4)) return set_error(RA_ERR_ALIGNMENT, "block_table, seq_lens and cu_new must be 4-byte aligned");
    }
    if (workspace_bytes < RA_WORKSPACE_MIN_BYTES)
        return set_error(RA_ERR_INVALID_ARG, "workspace smaller than RA_WORKSPACE_MIN_BYTES");
    AppendArgs a{};
    a.seqs.table = block_table;
    a.seqs.seq_lens = seq_lens;
    a.seqs.cu_q = cu_new;
    a.seqs.n_seqs = (int)n_seqs;
    a.seqs.T = (int)T;
    a.seqs.max_pages = (int)max_pages;
    a.seqs.page = (int)page_size;
    a.seqs.n_pages = (int)n_pages;
    a.k_new = static_cast<const uint4 *>(k_new);
    a.v_new = static_cast<const uint4 *>(v_new);
    a.k_pages = static_cast<uint4 *>(k_pages);
    a.v_pages = static_cast<uint4 *>(v_pages);
    a.new_stride = new_stride / 8;
    a.page_stride = page_stride / 8;
    a.pieces = (int)(H_kv * d / 8);
    a.status = static_cast<unsigned *>(workspace);
    // about two rounds of the unrolled copy to a block, fewer tokens where that leaves SMs idle
    int64_t per = 2 * 4 * kAppendThreads / a.pieces;
    if (per > T / (2 * kSms)) per = T / (2 * kSms);
    a.tokens = (int)(per < 1 ? 1 : per > kAppendTokens ? kAppendTokens : per);
    const int64_t blocks = (T + a.tokens - 1) / a.tokens;
    return launched(launch_dependent(paged_append_kernel, (unsigned)blocks, kAppendThreads, 0,
                                     static_cast<cudaStream_t>(stream), a));
}

}  // extern "C"
