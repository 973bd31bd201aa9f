// ra_warp_mma.cuh -- the warp-level pieces of the kernels whose tiles are too
// small for tcgen05: 16-byte asynchronous copies, ldmatrix, m16n8k16 products,
// and 16 rows by 16 keys of attention on them.
//
// A chunk is 16 keys (or their values) of D columns in shared memory, rows of
// 2 D bytes, the 16-byte piece c of row r at piece c ^ (r & 7), so that the
// eight rows an ldmatrix reads together lie in eight bank groups.
#pragma once
#include <cstdint>

#include "ra_device.cuh"

namespace ra {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// MT x 16 rows of one warp: Q fragments in, the running softmax and O.
// Lane (g = lane / 4, t4 = lane % 4) holds rows g and g + 8 of each 16, columns
// 2 t4, 2 t4 + 1 of each 8.
template <int D, int MT>
struct WarpRows {
    static constexpr int KS = D / 16;
    uint32_t q[MT][KS][4];
    float acc[MT][D / 8][4];
    float m[MT][2], l[MT][2];     // reference (log2 units) and this lane's share of the sum

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[mt][n][e] = 0.f;
            m[mt][0] = m[mt][1] = -INFINITY;
            l[mt][0] = l[mt][1] = 0.f;
        }
    }

    // One chunk: keys at sk, values at sv.  `whole`: every row sees all of it;
    // otherwise seen(mt, h) gives a row's visible columns as bits.
    template <class Seen>
    __device__ __forceinline__ void chunk(uint32_t sk, uint32_t sv, float scale_log2, bool whole, int lane, Seen seen) {
        const int t4 = lane & 3;
        float sc[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[mt][n][e] = 0.f;
        {
            // matrices: keys 0-7 / 8-15 by d 0-7 / 8-15 of the k-step
            const int kk = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
            const uint32_t row = sk + kk * (D * 2);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t b[4];
                ldmatrix4(b, row + (((ks * 2 + half) ^ (kk & 7)) << 4));
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    mma16816(sc[mt][0], q[mt][ks], b[0], b[1]);
                    mma16816(sc[mt][1], q[mt][ks], b[2], b[3]);
                }
            }
        }
        bool raise = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t bits = whole ? 0xffffu : seen(mt, h);
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = sc[mt][n][2 * h + e] * scale_log2;
                        if (!whole && !((bits >> (n * 8 + 2 * t4 + e)) & 1u)) x = -INFINITY;
                        sc[mt][n][2 * h + e] = x;
                        raise = raise || x > m[mt][h] + 8.f;
                    }
            }
        // The reference m of a row moves only when a score passes it by 2^8 (at
        // the row's first key, then rarely): exponentials stay below 2^8 and
        // their sums far inside 32 bits.
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x = fmaxf(fmaxf(sc[mt][0][2 * h], sc[mt][0][2 * h + 1]),
                                    fmaxf(sc[mt][1][2 * h], sc[mt][1][2 * h + 1]));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                    const float m_new = fmaxf(m[mt][h], x);
                    const float f = m[mt][h] > -INFINITY ? ex2(m[mt][h] - m_new) : 0.f;
                    m[mt][h] = m_new;
                    l[mt][h] *= f;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        acc[mt][n][2 * h] *= f;
                        acc[mt][n][2 * h + 1] *= f;
                    }
                }
        }
        // P as the sum of two bf16 values, about 16 bits: the output's own
        // rounding is the only one that shows
        uint32_t hi[MT][4], lo[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float ref = m[mt][h] > -INFINITY ? m[mt][h] : 0.f;
                    const float p0 = ex2(sc[mt][n][2 * h] - ref), p1 = ex2(sc[mt][n][2 * h + 1] - ref);
                    l[mt][h] += p0 + p1;
                    const uint32_t top = pack_bf16x2(p0, p1);
                    hi[mt][2 * n + h] = top;
                    lo[mt][2 * n + h] = pack_bf16x2(p0 - __uint_as_float(top << 16),
                                                    p1 - __uint_as_float(top & 0xffff0000u));
                }
        {
            // matrices: keys 0-7 / 8-15 by d 0-7 / 8-15 of a pair of column tiles
            const int kk = (lane & 7) + (((lane >> 3) & 1) << 3), half = lane >> 4;
            const uint32_t row = sv + kk * (D * 2);
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
                uint32_t b[4];
                ldmatrix4_trans(b, row + (((n * 2 + half) ^ (kk & 7)) << 4));
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    mma16816(acc[mt][2 * n], hi[mt], b[0], b[1]);
                    mma16816(acc[mt][2 * n + 1], hi[mt], b[2], b[3]);
                    mma16816(acc[mt][2 * n], lo[mt], b[0], b[1]);
                    mma16816(acc[mt][2 * n + 1], lo[mt], b[2], b[3]);
                }
            }
        }
    }
};

// Columns of the 16 keys from k0 on that a row sees, as bits.
__device__ __forceinline__ uint32_t seen_bits(int lo, int hi, int slo, int shi, int k0) {
    return (low_bits(hi - k0) & ~low_bits(lo - k0)) | (low_bits(shi - k0) & ~low_bits(slo - k0));
}

}  // namespace ra
