// paged_checks.h -- what the calls on a paged cache check of their arguments.
#pragma once
#include <initializer_list>

#include "ra_internal.h"

namespace ra {

inline bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr int64_t kMostStride = (int64_t)1 << 39;     // elements; a tensor map's strides stay below 2^40 bytes

inline ra_status check_heads(int64_t H, int64_t H_kv, int d) {
    if (d != 64 && d != 128) return set_error(RA_ERR_UNSUPPORTED, "head dimension d must be 64 or 128");
    if (H_kv < 1 || H_kv > H || H % H_kv)
        return set_error(RA_ERR_SHAPE, "the key/value head count must divide the query head count");
    if (H / H_kv > 128) return set_error(RA_ERR_UNSUPPORTED, "at most 128 query heads per key/value head");
    if (H > (int64_t)1 << 16) return set_error(RA_ERR_UNSUPPORTED, "H beyond the supported range");
    return RA_OK;
}

inline ra_status check_cache(int64_t T, int64_t n_seqs, int64_t H_kv, int d, int64_t n_pages, int64_t page,
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

// Pointers that a call cannot do without: tensors on 16 bytes, whole numbers on 4.
inline ra_status check_pointers(std::initializer_list<const void *> tensors, std::initializer_list<const void *> ints) {
    for (const void *p : tensors) {
        if (!p) return set_error(RA_ERR_INVALID_ARG, "null pointer argument");
        if (!aligned(p, 16)) return set_error(RA_ERR_ALIGNMENT, "every tensor pointer must be 16-byte aligned");
    }
    for (const void *p : ints) {
        if (!p) return set_error(RA_ERR_INVALID_ARG, "null pointer argument");
        if (!aligned(p, 4)) return set_error(RA_ERR_ALIGNMENT, "the int32 and fp32 vectors must be 4-byte aligned");
    }
    return RA_OK;
}

// T rows of `width` elements (of 2 bytes), `stride` apart.
struct TokenRows {
    const void *at;
    int64_t stride, width;
};
// Whether a row of x and a row of y share an element; rows no wider than their strides.
inline bool rows_meet(const TokenRows &x, const TokenRows &y, int64_t T) {
    using Wide = __int128;       // (the largest T and strides reach 2^63 between them)
    const int64_t a = (int64_t)(reinterpret_cast<uintptr_t>(x.at) / 2), b = (int64_t)(reinterpret_cast<uintptr_t>(y.at) / 2);
    if (a + (Wide)(T - 1) * x.stride + x.width <= b || b + (Wide)(T - 1) * y.stride + y.width <= a) return false;
    if (T == 1) return true;
    if (x.stride == y.stride) {
        // y's row j begins in x's row j + k or behind it (`in` elements from where that row does), before row j + k + 1
        int64_t k = (b - a) / x.stride, in = (b - a) % x.stride;
        if (in < 0) in += x.stride, --k;
        return (in < x.width && -T < k && k < T) || (in + y.width > x.stride && -T < k + 1 && k + 1 < T);
    }
    for (int64_t i = 0; i < T; ++i) {
        // the last row of y that begins before this row of x ends
        const Wide from = a + (Wide)i * x.stride, to = from + x.width;
        if (to <= b) continue;
        Wide j = (to - 1 - b) / y.stride;
        if (j > T - 1) j = T - 1;
        if (b + j * y.stride + y.width > from) return true;
    }
    return false;
}

}  // namespace ra
