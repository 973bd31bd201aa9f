// paged_keep.cu -- keeping the accepted path of a tree of drafted tokens in a
// paged cache.
//
// The tree's nodes lie behind the sequence's c other tokens in the order of
// their numbers; of them stay the path a_0 < a_1 < .. < a_{m-1} from a root to
// the last accepted node, moved to the places c, c + 1, .. c + m - 1, in every
// layer.  Since a_j >= j, and a_j > j for all later ones once it holds for one, a
// prefix stays where it is and every other node moves down: taken in
// order, a place is read before it is written.  One thread moves one 16-byte piece of the
// tokens of one layer's keys or values, eight at a time: the loads of a batch
// come before its stores, and later nodes lie behind the places it writes.
//
// Bound by the bytes of the nodes that move, read and written, and for few of
// them by the latency of a chain: lengths, parents, the walk up the tree, the
// table, the tokens.
#include "paged_checks.h"
#include "ra_device.cuh"
#include "ra_launch.h"
#include "ra_paged.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256, kBatch = 8, kSms = 152;

struct KeepArgs {
    PagedSeqs seqs;
    const int *last;
    int *new_lens, *path;
    uint4 *k, *v;
    int64_t page_stride, layer_stride;     // in 16-byte pieces
    int pieces, groups;                    // pieces of a token; blocks of a sequence
    int page_shift;                        // log2 of the page size
    int64_t items, per;                    // pieces of a token in all layers' keys and values; of a block
    unsigned *status;
};

__global__ void __launch_bounds__(kThreads) paged_keep_kernel(const KeepArgs a) {
    const PagedSeqs &sq = a.seqs;
    __shared__ short parents[kTreeMost], chain[kTreeMost];     // chain: the path from its end up
    __shared__ int64_t from[kTreeMost], to[kTreeMost];         // moved nodes' pieces in the pool
    __shared__ int pages[kTreeMost / 16 + 1];                  // of the places behind `before`
    __shared__ int s_m, s_stay;
    pdl_wait();
    const int s = blockIdx.x / a.groups, group = blockIdx.x % a.groups;
    const int c0 = paged_bound(sq, s), c1 = paged_bound(sq, s + 1);
    const int n_new = max(c1 - c0, 0), n = min(n_new, kTreeMost);
    const int last = a.last[s], len = sq.seq_lens[s];
    const int64_t before = (int64_t)len - n_new;
    bool bad = n_new > kTreeMost || before < 0 || last < -1 || last >= n || len > (int64_t)sq.max_pages * sq.page;
    const bool none = last < 0 || last >= n || before < 0;
    if (!none)
        for (int i = threadIdx.x; i <= last; i += kThreads) parents[i] = (short)tree_parent(sq.parents, c0, i, bad);
    // (the table beside the parents: one latency, and no entry without a place of the tree's)
    const int64_t page0 = before >> a.page_shift;
    if (!none)
        for (int64_t i = threadIdx.x; page0 + i <= (before + last) >> a.page_shift; i += kThreads)
            pages[i] = page0 + i < sq.max_pages ? sq.table[(size_t)s * sq.max_pages + page0 + i] : -1;
    __syncthreads();
    if (threadIdx.x == 0) {
        int m = 0;
        for (int p = none ? -1 : last; p >= 0; p = parents[p]) chain[m++] = (short)p;
        s_m = m;
        int stay = 0;
        while (stay < m && chain[m - 1 - stay] == stay) ++stay;
        s_stay = stay;
        if (group == 0) a.new_lens[s] = (int)max(before, (int64_t)0) + m;
    }
    __syncthreads();
    const int m = s_m, stay = s_stay, moved = m - stay;
    if (group == 0 && a.path)
        for (int i = threadIdx.x; i < n_new; i += kThreads) a.path[c0 + i] = i < m ? c0 + chain[m - 1 - i] : -1;
    auto place = [&](int64_t pos) -> int64_t {
        const int id = pages[(pos >> a.page_shift) - page0];
        if ((unsigned)id < (unsigned)sq.n_pages) return (int64_t)id * a.page_stride + (pos & (sq.page - 1)) * a.pieces;
        bad = true;
        return -1;
    };
    for (int i = threadIdx.x; i < moved; i += kThreads) {
        const int64_t src = place(before + chain[moved - 1 - i]), dst = place(before + stay + i);
        from[i] = dst < 0 ? -1 : src;
        to[i] = dst;
    }
    if (bad) atomicOr(a.status, RA_DEV_PAGE_BIT);
    __syncthreads();
    const int64_t end = min((group + 1) * a.per, a.items);
    for (int64_t e = group * a.per + threadIdx.x; e < end; e += kThreads) {
        const int64_t which = e / a.pieces;      // 2 * layer, + 1: values
        uint4 *pool = (which & 1 ? a.v : a.k) + (which >> 1) * a.layer_stride + (e - which * a.pieces);
        for (int j0 = 0; j0 < moved; j0 += kBatch) {
            uint4 x[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (j0 + j < moved && from[j0 + j] >= 0) x[j] = pool[from[j0 + j]];
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (j0 + j < moved && from[j0 + j] >= 0) pool[to[j0 + j]] = x[j];
        }
    }
}

}  // namespace
}  // namespace ra

extern "C" ra_status ra_paged_keep_path(void *k_pages, void *v_pages, const int32_t *block_table, const int32_t *seq_lens,
                                        const int32_t *cu_new, const int32_t *parents, const int32_t *last,
                                        int32_t *new_lens, int32_t *path, int64_t T, int64_t n_seqs, int64_t n_layers,
                                        int64_t H_kv, int d, int64_t n_pages, int64_t page_size, int64_t page_stride,
                                        int64_t layer_stride, int64_t max_pages, void *workspace, size_t workspace_bytes,
                                        void *stream) {
    using namespace ra;
    ra_status st = check_heads(H_kv, H_kv, d);
    if (st != RA_OK) return st;
    if ((st = check_cache(T, n_seqs, H_kv, d, n_pages, page_size, page_stride, max_pages)) != RA_OK) return st;
    if (n_layers < 0) return set_error(RA_ERR_SHAPE, "sizes must be non-negative");
    if (n_layers > 65536) return set_error(RA_ERR_UNSUPPORTED, "n_layers beyond the supported range");
    if (n_layers > 1) {
        if (layer_stride < 0 || layer_stride >= (int64_t)1 << 48)
            return set_error(RA_ERR_UNSUPPORTED, "layer_stride beyond the supported range");
        if (layer_stride % 8) return set_error(RA_ERR_ALIGNMENT, "layer_stride must be a multiple of 8 elements (16 bytes)");
        // layers one after another, or side by side within a page's stride
        const double one = (double)(page_size * H_kv * d), pool = (double)(n_pages - 1) * (double)page_stride + one;
        if ((double)layer_stride < pool && (double)page_stride < (double)(n_layers - 1) * (double)layer_stride + one)
            return set_error(RA_ERR_SHAPE, "layer_stride: pages of two layers would overlap");
        if ((double)layer_stride < one) return set_error(RA_ERR_SHAPE, "layer_stride: pages of two layers would overlap");
    }
    if (n_seqs == 0) return RA_OK;
    if ((st = check_pointers({workspace}, {seq_lens, cu_new, last, new_lens})) != RA_OK) return st;
    if (!aligned(path, 4)) return set_error(RA_ERR_ALIGNMENT, "the int32 and fp32 vectors must be 4-byte aligned");
    if (T > 0) {
        // (the path is walked and its pages looked up without layers too)
        if (n_pages == 0 || max_pages == 0) return set_error(RA_ERR_SHAPE, "new tokens need pages to lie in");
        if ((st = check_pointers({}, {block_table, parents})) != RA_OK) return st;
        if (n_layers > 0 && (st = check_pointers({k_pages, v_pages}, {})) != RA_OK) return st;
    }
    // a sequence's blocks read what the call is given all along
    const struct Words { const int32_t *at; int64_t n; } out[] = {{new_lens, n_seqs}, {path, path ? T : 0}},
        in[] = {{seq_lens, n_seqs}, {cu_new, n_seqs + 1}, {last, n_seqs}, {parents, T}, {block_table, n_seqs * max_pages}};
    auto meet = [](const Words &x, const Words &y) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(x.at), b = reinterpret_cast<uintptr_t>(y.at);
        return x.n > 0 && y.n > 0 && a < b + 4 * (uintptr_t)y.n && b < a + 4 * (uintptr_t)x.n;
    };
    for (const Words &x : out)
        for (const Words &y : in)
            if (meet(x, y)) return set_error(RA_ERR_INVALID_ARG, "new_lens and path must not overlap what the call reads");
    if (meet(out[0], out[1])) return set_error(RA_ERR_INVALID_ARG, "new_lens and path must not overlap");
    if (workspace_bytes < RA_WORKSPACE_MIN_BYTES)
        return set_error(RA_ERR_INVALID_ARG, "workspace smaller than RA_WORKSPACE_MIN_BYTES");
    KeepArgs a{};
    a.seqs.table = block_table;
    a.seqs.seq_lens = seq_lens;
    a.seqs.cu_q = cu_new;
    a.seqs.parents = parents;
    a.seqs.n_seqs = (int)n_seqs;
    a.seqs.T = (int)T;
    a.seqs.max_pages = (int)max_pages;
    a.seqs.page = (int)page_size;
    a.seqs.n_pages = (int)n_pages;
    a.last = last;
    a.new_lens = new_lens;
    a.path = path;
    a.k = static_cast<uint4 *>(k_pages);
    a.v = static_cast<uint4 *>(v_pages);
    a.page_stride = page_stride / 8;
    a.layer_stride = layer_stride / 8;
    a.pieces = (int)(H_kv * d / 8);
    a.items = n_layers * 2 * a.pieces;
    while ((int64_t)1 << a.page_shift < page_size) ++a.page_shift;
    a.status = static_cast<unsigned *>(workspace);
    // a piece to a thread while the blocks are few, more where sequences fill the SMs
    int64_t groups = (a.items + kThreads - 1) / kThreads;
    const int64_t most = (8 * kSms + n_seqs - 1) / n_seqs;
    if (groups > most) groups = most;
    if (groups < 1) groups = 1;
    a.groups = (int)groups;
    a.per = (a.items + groups - 1) / groups;
    if (n_seqs * groups > 0x7fffffffLL) return set_error(RA_ERR_UNSUPPORTED, "too many blocks for one launch");
    return launched(launch_dependent(paged_keep_kernel, (unsigned)(n_seqs * groups), kThreads, 0, static_cast<cudaStream_t>(stream), a));
}
