// kv_tile.cuh -- how a 128-row tile lies in shared memory, and clearing its tail.
#pragma once
#include <cstdint>

#include "ra_device.cuh"

namespace ra {

// How a K or V tile lies in its slot: eight rows of 128 bytes (64 columns) are
// 1024 bytes; kGroup is the distance from one such group of rows to the next,
// kHalf from columns 0-63 to 64-127.  A 2-D box per half gives all groups of a
// half in a row.  Paged tiles at d = 128 interleave the halves, so that one box
// brings a page's rows whole: half the copies of a tile of small pages (32 of
// 2 KB at 16 tokens a page otherwise, whose issue held the tile back by 0.5 us).
template <int D, bool INTERLEAVED>
struct KvTile {
    static constexpr uint32_t kGroup = INTERLEAVED ? 2048 : 1024;
    static constexpr uint32_t kHalf = INTERLEAVED ? 1024 : 128 * 128;
    static constexpr uint32_t kH = kHalf >> 4;            // descriptor units
    static constexpr uint32_t kStep = 2 * kGroup >> 4;    // 16 rows
};

// Zero rows [from, 128) of a tile in shared memory (nothing for from >= 128), by
// one warp before it issues the products that read them: what lies behind the
// last token may hold anything, NaN too, which a weight of 0 would not remove.
template <int D, class Tile>
__device__ __forceinline__ void zero_rows(uint32_t tile, int from, int lane) {
    if (from >= 128) return;
    for (int e = max(from, 0) * 8 + lane; e < 128 * 8; e += 32)
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                             tile + c * Tile::kHalf + (e >> 6) * Tile::kGroup + (e & 63) * 16),
                         "r"(0)
                         : "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

}  // namespace ra
