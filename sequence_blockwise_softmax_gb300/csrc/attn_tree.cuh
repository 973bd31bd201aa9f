// attn_tree.cuh -- attention of trees of new tokens over a paged cache on the
// sm_103a tensor cores, for more rows than the few-row form takes.
//
// A unit is up to 256 rows of one sequence and key/value head: the group's query
// heads of consecutive new tokens, packed token by token into 128-row Q tiles.
// It visits the 128-key tiles that its rows see, from the last down, so that
// each row walks its ancestors once, from itself up, and makes of those that lie
// in a tile the bits of their columns (TreeChain); all other keys are an interval
// and the sinks, as in the causal call.  S = Q K^T, P = 2^(S scale log2 e - m), O =
// sum P V with the softmax's reference and sums held in 32 bits as in
// attn_fwd_kernel.cuh; P is rounded to bf16 for the product and O divided by the
// sum of the rounded values.
//
// Most calls are bound by the cache's bytes: a key is used by a few dozen rows,
// and a CTA that ends at each unit leaves HBM idle for the 8 us of its start and
// end.  So CTAs stay, one to an SM, and take equal runs of a flat list of units'
// tiles; loads of the next unit are under way while the last one's rows go out.
// Up to eight key/value heads have a list each, cut alike, so that CTAs beside one
// another read the same tokens' heads, which lie side by side in HBM, at a time.
// A unit whose tiles lie in several runs leaves its pieces in the workspace, and a
// second kernel adds them.
//
// Warps (384 threads): 0 loads (TMA), 1 issues S, 3 issues PV, 2 finds the
// segments (pieces of units) of the CTA's run and posts them in a queue of two with their
// sequence's parents; 4-7 and 8-11 are two softmax groups, a thread to a row.
// Where units have two Q tiles (TWO) each group has one of them; where they have one
// (calls of at most 128 rows a unit) the groups take the key tiles in turn and add their
// rows at the end, which keeps both at work and halves the chain of a tile.
// One kernel for both kept their counts and slots in registers that the softmax
// lacks: 512 nodes over 32768 keys, 16 / 4 heads, 129 us at d = 128 and 102 at d = 64
// against 107 and 84 as two kernels.  (They spill up to 28 bytes all the same, the two-tile
// one at d = 64 none.)
#pragma once
#include "kv_tile.cuh"
#include "paged_launch.h"
#include "ra_device.cuh"
#include "ra_internal.h"
#include "ra_paged.cuh"
#include "ra_tree.cuh"

namespace ra {

struct TreeArgs {
    PagedSeqs seqs;             // unit_tokens: tokens of a unit
    int tile_tokens, page_box;  // tokens of a Q tile; keys of a copy
    int two;                    // units have two Q tiles (for the join: the main kernel is one for each)
    int min_run;                // tiles of a run at least
    int streams, heads;         // lists side by side, of this many key/value heads each
    float scale_log2;
    unsigned *status;
    void *o;
    float *lse;
    int o_bf16;
    // pieces of cut units, place 2 * CTA for one that began before, 2 * CTA + 1 for one that goes
    // on: each Q tile's rows [D / 4][128] (two places for them) and their (m, l, lr); and each CTA's TreeCut
    float4 *part_o, *part_ml;
    struct TreeCut *cuts;
};

// The unit that begins in a CTA's run and goes on through the next `more` runs: n
// tokens from t0 on, of key/value head hk; n = 0: there is none.
struct __align__(16) TreeCut {
    int t0, n, hk, more;
};

// A kernel in PARTS works on a segment by at most kTreePart (1024) tiles at a time, whose rows are added
// in fp32 where the segment's piece has its place in the workspace.  The tensor cores cut
// off what lies below 2^-21 of a sum that they add to, at each of a tile's eight products: where
// values are alike O comes out short by 3e-4 after 1024 tiles, by 5e-3 after 2^20 keys and by a quarter
// after 2^26.  It also keeps segments well inside the waits' limit of two seconds, which one
// of 2^28 keys passes.  The code costs d = 64 up to 5 % (500 nodes 43.8 to 45.9 us) and d = 128
// 0.3 %, so calls whose units cannot be longer (tree_in_parts) do without.
struct TreePart : TreeSegment {
    int earlier;            // the segment had parts before
    int left;               // its tiles behind this part
    __device__ __forceinline__ void take(int n) {
        tiles = min(n, kTreePart);
        left = n - tiles;
    }
};

// What goes through the queue of segments.
template <bool PARTS>
struct TreeQueued {
    using Type = TreeSegment;
};
template <>
struct TreeQueued<true> {
    using Type = TreePart;
};

template <int D, bool PARTS>
struct TreeSmem {
    static constexpr uint32_t kTile = 128u * D * 2u;     // 128 rows x d bf16
    static constexpr uint32_t kBox = 128u * 128u;        // 128 rows x 64 columns
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kP = 160u * 1024;          // P_g (d = 128), and where groups meet at a unit's end
    // K and V tiles lie between Q and P: 3 slots at d = 128 with two Q tiles, 4 with one, 8 at d = 64
    static constexpr int kMostSlots = 8;
    static __host__ __device__ constexpr uint32_t ring(bool two) { return two || D == 64 ? 2 * kTile : kTile; }
    static __host__ __device__ constexpr int slots(bool two) { return D == 64 ? 8 : two ? 3 : 4; }
    static constexpr uint32_t kBars = 224u * 1024;
    static constexpr int kNumBars = 2 + 3 * kMostSlots + 8 + 4 + 2 + 2;
    static constexpr uint32_t kSegs = (kBars + kNumBars * 8 + 15) / 16 * 16;
    static constexpr uint32_t kMisc = kSegs + 2 * sizeof(typename TreeQueued<PARTS>::Type);   // tensor memory's address, flags, the scan's sums
    static constexpr uint32_t kParents = kMisc + 128;
    static constexpr uint32_t kBytes = kParents + kTreeMost * 2;
};
static_assert(TreeSmem<128, true>::kBytes <= 232448, "what a CTA may have");

__device__ __forceinline__ void st_shared_f4(uint32_t addr, const float4 &x) {
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w) : "memory");
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
    float4 x;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(addr) : "memory");
    return x;
}
// The denominator's range in which the exponentials' reference stays (see
// attn_fwd_kernel.cuh).
constexpr float kTreeSumLo = 0x1p-32f, kTreeSumHi = 0x1p32f;

// Columns c0 .. c0 + 7 of a final row whose first element is `to`, and a row's LSE.
__device__ __forceinline__ void tree_store8(const TreeArgs &a, size_t to, int c0, const float (&x)[8], float inv) {
    if (a.o_bf16) {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o) + to + c0) =
            make_uint4(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv),
                       pack_bf16x2(x[4] * inv, x[5] * inv), pack_bf16x2(x[6] * inv, x[7] * inv));
    } else {
        float *dst = static_cast<float *>(a.o) + to + c0;
        *reinterpret_cast<float4 *>(dst) = make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
        *reinterpret_cast<float4 *>(dst + 4) = make_float4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
    }
}
__device__ __forceinline__ void tree_store_lse(const TreeArgs &a, size_t tok, int head, float top, float l) {
    if (a.lse) a.lse[(size_t)head * a.seqs.T + tok] = l > 0.f ? (top + lg2(l)) * 0.6931471805599453f : -INFINITY;
}

template <int D, bool TWO, bool PARTS>
__global__ void __launch_bounds__(384, 1)
    paged_tree_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv, const __grid_constant__ TreeArgs args) {
    using L = TreeSmem<D, PARTS>;
    using Queued = typename TreeQueued<PARTS>::Type;
    using KT = KvTile<D, D == 128>;
    constexpr int HALVES = D / 64, MOST = L::kMostSlots;
    constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 128, false), IDESC_O = idesc_bf16_f32(128, D, true);
    // at d = 64 tensor memory has room for P beside S and O
    constexpr bool P_IN_TMEM = D == 64;
    const PagedSeqs &sq = args.seqs;

    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t s_base = smem_u32(smem);
    if ((s_base & 1023u) != 0u) {
        pdl_wait();
        if (threadIdx.x == 0) {
            atomicOr(args.status, RA_DEV_SMEM_ALIGN_BIT);
            args.cuts[blockIdx.x] = TreeCut{0, 0, 0, 0};
        }
        return;
    }
    auto BAR = [&](int i) -> uint32_t { return s_base + L::kBars + 8u * (uint32_t)i; };
    constexpr int B_QFULL = 0, B_QFREE = 1, B_KF = 2, B_VF = B_KF + MOST, B_SLOTE = B_VF + MOST, B_SFULL = B_SLOTE + MOST,
                  B_SFREE = B_SFULL + 2, B_PFULL = B_SFREE + 2, B_PVDONE = B_PFULL + 2, B_SEGFULL = B_PVDONE + 2,
                  B_SEGFREE = B_SEGFULL + 2, B_PARFULL = B_SEGFREE + 2, B_PARFREE = B_PARFULL + 1, B_MEET = B_PARFREE + 1,
                  B_FINAL = B_MEET + 1;
    static_assert(B_FINAL + 1 == L::kNumBars, "one place for each barrier");
    Queued *segs = reinterpret_cast<Queued *>(smem + L::kSegs);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);
    long long *warp_sums = reinterpret_cast<long long *>(smem + L::kMisc + 16);      // 12
    long long *run_off = reinterpret_cast<long long *>(smem + L::kMisc + 112);
    int *run_seq = reinterpret_cast<int *>(smem + L::kMisc + 8);
    short *parents = reinterpret_cast<short *>(smem + L::kParents);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr bool two = TWO;
    constexpr int nsl = L::slots(two);
    const uint32_t ring = s_base + L::ring(two);
    // load i's slot, and how many loads that slot has had before.  (Both depend on TWO alone: as
    // divisions by a variable they held up loads and products, 64 sequences of 500-12000
    // keys 296 us against 287.)
    auto round_of = [](unsigned i) -> unsigned { return i / nsl; };
    auto slot_of = [](unsigned i) -> int { return (int)(i % nsl); };

    // ---- setup (nothing here reads what the kernel before may still write)
    if (threadIdx.x == 32) {
        mbar_init(BAR(B_QFULL), 1);
        mbar_init(BAR(B_QFREE), 1);
        for (int s = 0; s < MOST; ++s) {
            mbar_init(BAR(B_KF + s), 1);
            mbar_init(BAR(B_VF + s), 1);
            mbar_init(BAR(B_SLOTE + s), 1);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(BAR(B_SFULL + g), 1);
            mbar_init(BAR(B_SFREE + g), 128);
            mbar_init(BAR(B_PFULL + g), 128);
            mbar_init(BAR(B_PVDONE + g), 1);
            mbar_init(BAR(B_SEGFULL + g), 1);
            mbar_init(BAR(B_SEGFREE + g), 11);       // the warps that read it
        }
        mbar_init(BAR(B_PARFULL), 32);
        mbar_init(BAR(B_PARFREE), 8);
        mbar_init(BAR(B_MEET), 8);
        mbar_init(BAR(B_FINAL), 2);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    if (warp == 2) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    pdl_wait();

    // ---- the CTA's run, places [pos, end) of the flat list, and where it begins; warp 2
    // goes on from there
    const int run = blockIdx.x / args.streams, runs = gridDim.x / args.streams;
    const int head0 = (blockIdx.x - run * args.streams) * args.heads;     // the stream's heads
    long long pos = 0, end = 0, per = 1, off = 0, head_cost = 1;
    int pad = 1;
    TreeSeq seq{};
    if (sq.n_seqs > 32) {
        // consecutive sequences to a thread, and the sum of what lies before them
        const int each = (sq.n_seqs + 383) / 384;
        const int s0 = min((int)threadIdx.x * each, sq.n_seqs), s1 = min(s0 + each, sq.n_seqs);
        long long mine = 0, total = 0;
        for (int s = s0; s < s1; ++s) {
            mine += tree_head_cost(sq, tree_seq(sq, s)) * args.heads;
            if (blockIdx.x == 0 && paged_bad_counts(sq, s)) atomicOr(args.status, RA_DEV_PAGE_BIT);
        }
        long long inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += up;
        }
        if (lane == 31) warp_sums[warp] = inc;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 12; ++w) {
            if (w < warp) inc += warp_sums[w];
            total += warp_sums[w];
        }
        per = tree_per(total, runs, args.min_run, two);
        pos = run * per;
        end = min(pos + per, total);
        if (inc - mine <= pos && pos < inc) {
            long long rest = pos - (inc - mine);
            int s = s0;
            for (long long c; s + 1 < s1 && rest >= (c = tree_head_cost(sq, tree_seq(sq, s)) * args.heads); ++s) rest -= c;
            *run_seq = s;
            *run_off = rest;
        }
        __syncthreads();
        if (warp == 2 && pos < end) {
            off = *run_off;
            seq = tree_seq(sq, *run_seq);
            head_cost = tree_head_cost(sq, seq);
        }
    } else if (warp == 2) {
        // a sequence to a lane
        const TreeSeq t = tree_seq(sq, min(lane, sq.n_seqs - 1));
        if (blockIdx.x == 0 && paged_bad_counts(sq, t.s)) atomicOr(args.status, RA_DEV_PAGE_BIT);
        const int units = (int)__reduce_add_sync(0xffffffffu, lane < sq.n_seqs ? (unsigned)t.blocks : 0u);
        long long of_head, mine, inc, total;
#pragma unroll 1
        while (true) {
            of_head = lane < sq.n_seqs ? tree_head_cost(sq, t, pad) : 0;
            mine = inc = of_head * args.heads;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long up = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += up;
            }
            total = __shfl_sync(0xffffffffu, inc, 31);
            if (pad > 1) break;
            per = tree_per(total, runs, args.min_run, two);
            pad = tree_pad((long long)units * args.heads, total, runs, per, two ? 1 : 2);
            if (pad == 1) break;
            per = pad;
        }
        pos = run * per;
        end = min(pos + per, total);
        const unsigned found = __ballot_sync(0xffffffffu, inc - mine <= pos && pos < inc);
        const int at = found ? __ffs(found) - 1 : 0;
        off = pos - __shfl_sync(0xffffffffu, inc - mine, at);
        seq.s = at;
        seq.c0 = __shfl_sync(0xffffffffu, t.c0, at);
        seq.c1 = __shfl_sync(0xffffffffu, t.c1, at);
        seq.len = __shfl_sync(0xffffffffu, t.len, at);
        seq.blocks = __shfl_sync(0xffffffffu, t.blocks, at);
        head_cost = __shfl_sync(0xffffffffu, of_head, at);
    }
    if (warp == 2) {
        Queued e{};
        e.tiles = -1;
        if (pos < end) {
            static_cast<TreeSegment &>(e) = tree_first_segment(sq, seq, head_cost, head0, off, pos, end, per, run, pad);
            if constexpr (PARTS) e.take(e.tiles);
        }
        if (lane == 0) segs[0] = e;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (segs[0].tiles < 0) {                 // more CTAs than runs
        if (threadIdx.x == 0) args.cuts[blockIdx.x] = TreeCut{0, 0, 0, 0};
        if (warp == 2) tmem_dealloc(tmem, 512);
        return;
    }

    auto timed_out = [&]() {
        if (lane == 0) {
            *abort_flag = 1;
            atomicOr(args.status, RA_DEV_TIMEOUT_BIT);
        }
    };
    // segment number `seg` once it is posted; false at the queue's end (or after a timeout: ok false)
    auto next_segment = [&](int seg, TreeSegment &e, bool &ok) -> bool {
        ok = seg == 0 || warp_wait(BAR(B_SEGFULL + (seg & 1)), (seg >> 1) & 1, abort_flag);   // (the first is there)
        if (!ok) return false;
        e = segs[seg & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_SEGFREE + (seg & 1)));
        return e.tiles >= 0;
    };
    auto walk_of = [](const TreeSegment &e) {
        TreeWalk w;
        w.i = e.i0;
        w.end = e.i0 + e.tiles;
        w.n_main = e.n_main;
        w.last = e.last;
        w.s0 = e.s0;
        w.seek();
        return w;
    };
    // K and V tiles go to the slots in the order K(0), K(1), V(0), K(2), V(1), ..
    // over all segments: K(t) is load 2 t - 1 (K(0) load 0), V(t) load 2 t + 2 (at a
    // segment's end that one goes first, and at the last one's the other is left out).
    auto k_load = [](int t) { return t == 0 ? 0 : 2 * t - 1; };
    auto v_load = [](int t) { return 2 * t + 2; };

    if (warp == 0) {
        // ================================================= loads
        regs_shrink<56>();
        uint32_t k_loads = 0, v_loads = 0;   // bit s: slot s has had a load of the kind, bit 8 + s: the parity of its last
        auto load = [&](unsigned i, int page, int tile, int head, bool is_k) -> bool {
            const int sl = slot_of(i);
            if (i >= (unsigned)nsl && !warp_wait(BAR(B_SLOTE + sl), (round_of(i) - 1) & 1, abort_flag)) return false;
            const uint32_t full = BAR((is_k ? B_KF : B_VF) + sl);
            uint32_t &loads = is_k ? k_loads : v_loads;
            loads = (loads & (1u << sl)) ? loads ^ (256u << sl) : loads | (1u << sl);
            if (lane == 0) mbar_arrive_expect_tx(full, L::kTile);
            __syncwarp();
            if (lane * args.page_box < 128) {
                const int y = (tile * 128 + lane * args.page_box) & (sq.page - 1);
                const uint32_t to = ring + sl * L::kTile + (lane * args.page_box >> 3) * KT::kGroup;
                if constexpr (HALVES == 2) tma_load_5d(to, is_k ? &tmk : &tmv, full, 0, 0, 2 * head, y >> 3, page);
                else tma_load_3d(to, is_k ? &tmk : &tmv, full, head * D, y, page);
            }
            __syncwarp();
            return true;
        };
        bool ok = true;
        int t = 0, q_loads = 0;
        int v_page = 0, v_tile = 0, v_head = 0;
        TreeSegment e;
        for (int seg = 0; ok && next_segment(seg, e, ok); ++seg) {
            // lane i's page of a key tile (its box of page_box keys), or one past
            // the last page, which reads as zeros, where no row sees any of its keys
            const RowKeys first = paged_row(sq, e.before);
            const int last_hi = e.before + e.first + e.n;
            auto page_of = [&](int tile) -> int {
                int z = sq.n_pages;
                const int k0 = tile * 128 + lane * args.page_box;
                if (lane * args.page_box < 128 && paged_needed(first, last_hi, e.len, k0, args.page_box)) {
                    z = sq.table[(size_t)e.s * sq.max_pages + k0 / sq.page];
                    if ((unsigned)z >= (unsigned)sq.n_pages) {
                        atomicOr(args.status, RA_DEV_PAGE_BIT);
                        z = sq.n_pages;
                    }
                }
                return z;
            };
            TreeWalk w = walk_of(e);
            int page = w.valid() ? page_of(w.tile) : 0;
            for (int j = 0; ok && w.valid(); ++j) {
                if (!(ok = load(k_load(t), page, w.tile, e.hk, true))) break;
                if (j > 0 && !(ok = load(v_load(t - 1), v_page, v_tile, v_head, false))) break;
                if (j == 0) {
                    // Q once the last segment's products have read theirs
                    if (q_loads > 0 && !(ok = warp_wait(BAR(B_QFREE), (q_loads - 1) & 1, abort_flag))) break;
                    if (lane == 0) {
                        const int tiles = two && e.n > args.tile_tokens ? 2 : 1;
                        mbar_arrive_expect_tx(BAR(B_QFULL), tiles * HALVES * args.tile_tokens * sq.group * 128);
                        for (int g = 0; g < tiles; ++g)
                            for (int c = 0; c < HALVES; ++c)
                                tma_load_3d(s_base + L::kQ + g * L::kTile + c * L::kBox, &tmq, BAR(B_QFULL), 64 * c,
                                            e.hk * sq.group, e.t0 + g * args.tile_tokens);
                    }
                    __syncwarp();
                    ++q_loads;
                }
                v_page = page;
                v_tile = w.tile;
                v_head = e.hk;
                ++t;
                w.next();
                if (w.valid()) page = page_of(w.tile);      // (read a tile ahead)
            }
            // the last V does not wait for the next segment, whose pages are read first (and
            // which may have no tile)
            if (ok && e.tiles > 0) ok = load(v_load(t - 1), v_page, v_tile, v_head, false);
        }
        if (!ok) {
            timed_out();
            // let the copies already issued land before the CTA exits
            volatile int never = 0;
            if (q_loads > 0) mbar_wait(BAR(B_QFULL), (q_loads - 1) & 1, &never);
            for (int sl = 0; sl < nsl; ++sl) {
                if ((k_loads >> sl) & 1u) mbar_wait(BAR(B_KF + sl), (k_loads >> (8 + sl)) & 1u, &never);
                if ((v_loads >> sl) & 1u) mbar_wait(BAR(B_VF + sl), (v_loads >> (8 + sl)) & 1u, &never);
            }
        }
    } else if (warp == 1) {
        // ================================================= S products
        regs_shrink<56>();
        const uint64_t dq0 = sdesc_sw128(s_base + L::kQ, 16, 1024), dq1 = sdesc_sw128(s_base + L::kQ + L::kTile, 16, 1024);
        const uint64_t dk0 = sdesc_sw128(ring, 16, KT::kGroup);
        auto issue_s = [&](int g, uint64_t a0, int slot) {
            const uint64_t b0 = dk0 + (uint64_t)(slot * (L::kTile >> 4));
            const uint32_t d = tmem + g * 128;
            mma_ss_elect<0, 0>(d, a0, b0, IDESC_S, 0u);
            mma_ss_elect<2, 2>(d, a0, b0, IDESC_S, 1u);
            mma_ss_elect<4, 4>(d, a0, b0, IDESC_S, 1u);
            mma_ss_elect<6, 6>(d, a0, b0, IDESC_S, 1u);
            if (D == 128) {
                constexpr uint32_t h = L::kBox >> 4, kh = KT::kH;
                mma_ss_elect<h, kh>(d, a0, b0, IDESC_S, 1u);
                mma_ss_elect<h + 2, kh + 2>(d, a0, b0, IDESC_S, 1u);
                mma_ss_elect<h + 4, kh + 4>(d, a0, b0, IDESC_S, 1u);
                mma_ss_elect<h + 6, kh + 6>(d, a0, b0, IDESC_S, 1u);
            }
            tc_commit_elect(BAR(B_SFULL + g));
        };
        uint32_t k_parity = 0;   // bit s: parity of the next K load of slot s
        int n0 = 0, n1 = 0;      // products issued per group
        bool ok = true;
        int t = 0, q_loads = 0;
        TreeSegment e;
        for (int seg = 0; ok && next_segment(seg, e, ok); ++seg) {
            const int tiles = e.tiles;
            const bool second = e.n > args.tile_tokens;      // two: there is a second Q tile
            if (tiles > 0) ok = warp_wait(BAR(B_QFULL), q_loads++ & 1, abort_flag);
#pragma unroll 1
            for (int j = 0; ok && j < tiles; ++j, ++t) {
                const int sl = slot_of(k_load(t));
                ok = warp_wait(BAR(B_KF + sl), (k_parity >> sl) & 1u, abort_flag);
                k_parity ^= 1u << sl;
                if (!ok) break;
                if (two || !(j & 1)) {
                    if (n0 > 0 && !(ok = warp_wait(BAR(B_SFREE + 0), (n0 - 1) & 1, abort_flag))) break;
                    tc_fence_after();
                    issue_s(0, dq0, sl);
                    ++n0;
                    __syncwarp();
                }
                if (two ? second : (j & 1)) {
                    if (n1 > 0 && !(ok = warp_wait(BAR(B_SFREE + 1), (n1 - 1) & 1, abort_flag))) break;
                    tc_fence_after();
                    issue_s(1, two ? dq1 : dq0, sl);
                    ++n1;
                }
                tc_commit_elect(BAR(B_SLOTE + sl));
                __syncwarp();
            }
            if (ok && tiles > 0) tc_commit_elect(BAR(B_QFREE));
        }
        if (!ok) timed_out();
        // every product this warp issued has finished before tensor memory is freed
        __syncwarp();
        tc_commit_elect(BAR(B_FINAL));
        __syncwarp();
        volatile int never = 0;
        mbar_wait(BAR(B_FINAL), 0, &never);
    } else if (warp == 3) {
        // ================================================= PV products
        regs_shrink<56>();
        const uint64_t dp0 = sdesc_sw128(s_base + L::kP, 16, 1024), dp1 = sdesc_sw128(s_base + L::kP + 2 * L::kBox, 16, 1024);
        const uint64_t dv0 = sdesc_sw128(ring, KT::kHalf, KT::kGroup);
        auto issue_pv = [&](int g, uint64_t a0, int slot, bool first) {
            const uint64_t b0 = dv0 + (uint64_t)(slot * (L::kTile >> 4));
            const uint32_t d = tmem + 256 + g * D;
            constexpr uint32_t vs = KT::kStep, hb = L::kBox >> 4;
            if constexpr (P_IN_TMEM) {
                const uint32_t p = tmem + 384 + g * 64;      // 16 keys are 8 packed columns
                mma_ts_elect<0, 0>(d, p, b0, IDESC_O, first ? 0u : 1u);
                mma_ts_elect<8, vs>(d, p, b0, IDESC_O, 1u);
                mma_ts_elect<16, 2 * vs>(d, p, b0, IDESC_O, 1u);
                mma_ts_elect<24, 3 * vs>(d, p, b0, IDESC_O, 1u);
                mma_ts_elect<32, 4 * vs>(d, p, b0, IDESC_O, 1u);
                mma_ts_elect<40, 5 * vs>(d, p, b0, IDESC_O, 1u);
                mma_ts_elect<48, 6 * vs>(d, p, b0, IDESC_O, 1u);
                mma_ts_elect<56, 7 * vs>(d, p, b0, IDESC_O, 1u);
            } else {
                mma_ss_elect<0, 0>(d, a0, b0, IDESC_O, first ? 0u : 1u);
                mma_ss_elect<2, vs>(d, a0, b0, IDESC_O, 1u);
                mma_ss_elect<4, 2 * vs>(d, a0, b0, IDESC_O, 1u);
                mma_ss_elect<6, 3 * vs>(d, a0, b0, IDESC_O, 1u);
                mma_ss_elect<hb, 4 * vs>(d, a0, b0, IDESC_O, 1u);
                mma_ss_elect<hb + 2, 5 * vs>(d, a0, b0, IDESC_O, 1u);
                mma_ss_elect<hb + 4, 6 * vs>(d, a0, b0, IDESC_O, 1u);
                mma_ss_elect<hb + 6, 7 * vs>(d, a0, b0, IDESC_O, 1u);
            }
            tc_commit_elect(BAR(B_PVDONE + g));
        };
        uint32_t v_parity = 0;   // bit s: parity of the next V load of slot s
        int n0 = 0, n1 = 0;      // products issued per group
        bool ok = true;
        int t = 0;
        TreeSegment e;
        for (int seg = 0; ok && next_segment(seg, e, ok); ++seg) {
            const int tiles = e.tiles;
            const bool second = e.n > args.tile_tokens;
            TreeWalk w = walk_of(e);
#pragma unroll 1
            for (int j = 0; ok && j < tiles; ++j, ++t, w.next()) {
                const int sl = slot_of(v_load(t));
                ok = warp_wait(BAR(B_VF + sl), (v_parity >> sl) & 1u, abort_flag);
                v_parity ^= 1u << sl;
                if (!ok) break;
                // what lies behind the last token may be NaN, which a weight of 0 would not remove
                zero_rows<D, KT>(ring + sl * L::kTile, e.len - w.tile * 128, lane);
                if (two || !(j & 1)) {
                    if (!(ok = warp_wait(BAR(B_PFULL + 0), n0 & 1, abort_flag))) break;
                    tc_fence_after();
                    issue_pv(0, dp0, sl, j == 0);
                    ++n0;
                    __syncwarp();
                }
                if (two ? second : (j & 1)) {
                    if (!(ok = warp_wait(BAR(B_PFULL + 1), n1 & 1, abort_flag))) break;
                    tc_fence_after();
                    issue_pv(1, dp1, sl, j <= 1 - (int)two);
                    ++n1;
                }
                tc_commit_elect(BAR(B_SLOTE + sl));
                __syncwarp();
            }
        }
        if (!ok) timed_out();
        __syncwarp();
        tc_commit_elect(BAR(B_FINAL));
        __syncwarp();
        volatile int never = 0;
        mbar_wait(BAR(B_FINAL), 0, &never);
    } else if (warp == 2) {
        // ================================================= segments
        regs_shrink<56>();
        // The segment's parents, once the groups are done with those before.
        auto post_parents = [&](int seg, const TreeSegment &e) -> bool {
            if (seg > 0 && !warp_wait(BAR(B_PARFREE), (seg - 1) & 1, abort_flag)) return false;
            bool bad = false;
            const int c0 = e.t0 - e.first;
            for (int i = lane; i < e.first + e.n; i += 32) parents[i] = (short)tree_parent(sq.parents, c0, i, bad);
            if (bad) atomicOr(args.status, RA_DEV_PAGE_BIT);
            mbar_arrive(BAR(B_PARFULL));
            return true;
        };
        auto post = [&](int seg, const Queued &e) -> bool {
            if (seg >= 2 && !warp_wait(BAR(B_SEGFREE + (seg & 1)), ((seg >> 1) - 1) & 1, abort_flag)) return false;
            if (lane == 0) {
                segs[seg & 1] = e;
                mbar_arrive(BAR(B_SEGFULL + (seg & 1)));
            }
            __syncwarp();
            return e.tiles < 0 || post_parents(seg, e);
        };
        if (lane == 0) mbar_arrive(BAR(B_SEGFULL));      // (of the first segment)
        Queued e = segs[0];
        int seg = 1;
        bool ok = post_parents(0, e);
        TreeCut cut{0, 0, 0, 0};
        while (true) {
            if constexpr (PARTS)
                while (ok && e.left > 0) {
                    e.earlier = 1;
                    e.i0 += e.tiles;
                    e.take(e.left);
                    ok = post(seg++, e);
                }
            pos += e.places;
            if (!e.whole && e.begins) cut = TreeCut{e.t0, e.n, e.hk, e.more};
            if (!ok || pos >= end) break;
            static_cast<TreeSegment &>(e) = tree_next_segment(sq, seq, e, head0, args.heads, pos, end, per, run, pad);
            if constexpr (PARTS) {
                e.earlier = 0;
                e.take(e.tiles);
            }
            ok = post(seg++, e);
        }
        if (lane == 0) args.cuts[blockIdx.x] = cut;
        e.tiles = -1;
        if (ok) ok = post(seg, e);
        if (!ok) timed_out();
    } else {
        // ================================================= softmax
        regs_grow<224>();
        const int g = (warp - 4) >> 2, wq = warp & 3;
        const int r = wq * 32 + lane;                 // row of the Q tile (= tensor memory's lane)
        const int my_head = r % sq.group, my_tok = (two ? g * args.tile_tokens : 0) + r / sq.group;
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        const uint32_t tS = tmem + lane_off + g * 128, tO = tmem + lane_off + 256 + g * D;
        const float sl2 = args.scale_log2;
        int n = 0;                 // tiles this group has taken, in all segments
        int meets = 0;
        bool ok = true;
        // Both groups' threads meet: what they wrote before is seen after.  `owed`: this warp has
        // arrived and not waited yet.
        bool owed = false;
        auto arrive = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(B_MEET));
            owed = true;
        };
        auto settle = [&]() -> bool {
            if (owed) ok = warp_wait(BAR(B_MEET), meets++ & 1, abort_flag);
            owed = false;
            return ok;
        };
        // A segment's rows: what they see of the tokens before the new ones, their
        // chains, whether they are stored (others see what the last token sees, so that no
        // tile is masked for their sake).
        // (counted from the first new token)
        int see_lo = 0, see_sinks = 0;       // [see_lo, 0) and, of a window's sinks, all below see_sinks
        // The row's chain (TreeChain) and its bits in the last tile with new tokens.
        int chain_at = -1, chain_steps = 0, chain_far = 0;
        uint32_t drafted[4] = {0u, 0u, 0u, 0u};
        bool live = false;
        // (a segment's fields are read from shared memory as they are needed, to keep them
        // out of the tile loop's registers)
        auto begin = [&](int seg) -> bool {
            ok = seg == 0 || warp_wait(BAR(B_SEGFULL + (seg & 1)), (seg >> 1) & 1, abort_flag);
            const Queued &e = segs[seg & 1];
            if (!ok || e.tiles < 0 || !(ok = warp_wait(BAR(B_PARFULL), seg & 1, abort_flag))) return false;
            live = r / sq.group < args.tile_tokens && my_tok < e.n;
            const int node = e.first + min(my_tok, e.n - 1);
            int depth = 0;
            if (sq.window > 0)
                for (int p = parents[node]; p >= 0; p = parents[p]) ++depth;
            const RowKeys rk = tree_row(sq, e.before + depth, e.before);
            see_lo = rk.lo - e.before;
            see_sinks = rk.shi - e.before;
            TreeChain chain;
            chain.start(node, depth, e.before, sq.window, sq.sinks);
            chain_at = chain.at;
            chain_steps = chain.steps;
            chain_far = chain.far;
            return true;
        };
        bool more = begin(0);
        for (int seg = 0; ok && more; ++seg) {
            const Queued &e = segs[seg & 1];
            const bool warp_live = __any_sync(0xffffffffu, live);
            bool holds = true;        // the parents are still needed
            auto let_go = [&]() {
                __syncwarp();
                if (holds && lane == 0) mbar_arrive(BAR(B_PARFREE));
                holds = false;
            };
            float m_ref = 0.f, l = 0.f, lr = 0.f;   // reference (log2 units), sum, sum of the rounded weights
            int mine = 0;                           // tiles of this segment taken
            // The group's tiles j, and the first key of one, counted from the first new token.
            const int step = two ? 1 : 2, tiles_end = two && g == 1 && e.n <= args.tile_tokens ? 0 : e.tiles;
            int j = two ? 0 : g, first_new = tree_tile(e, j) * 128 - e.before;
            while (j < tiles_end) {
                if (holds && first_new + 128 <= 0) let_go();
                if (!(ok = warp_wait(BAR(B_SFULL + g), n & 1, abort_flag))) break;
                if (!warp_live) {
                    mbar_arrive(BAR(B_SFREE + g));
                    if (mine > 0 && !(ok = warp_wait(BAR(B_PVDONE + g), (n - 1) & 1, abort_flag))) break;
                    if (!settle()) break;
                    mbar_arrive(BAR(B_PFULL + g));
                    ++mine;
                    ++n;
                    j += step;
                    first_new = tree_tile(e, j) * 128 - e.before;
                    continue;
                }
                tc_fence_after();
                // columns [lim_lo, lim), the sinks up to sk_hi and the new tokens' bits are seen
                const int lim = -first_new, lim_lo = see_lo - first_new, sk_hi = see_sinks - first_new;
                const bool partial = lim < 128 || lim_lo > 0;
                bool any_drafted = false;
                if (holds) {
                    TreeChain chain;
                    chain.start(chain_at, 0, 0, sq.window, 0);
                    chain.steps = chain_steps;
                    chain.far = chain_far;
                    uint32_t word[4];
                    chain.tile(parents, first_new, word);
                    chain_at = chain.at;
                    chain_steps = chain.steps;
#pragma unroll
                    for (int q = 0; q < 4; ++q) drafted[q] = word[q];
                    any_drafted = (word[0] | word[1] | word[2] | word[3]) != 0u;
                }
                uint32_t sr[4][32];
                auto load_s = [&]() {
#pragma unroll
                    for (int q = 0; q < 4; ++q) tmem_ld32(tS + q * 32, sr[q]);
                    tmem_wait_ld();
                    if (__any_sync(0xffffffffu, partial)) {
                        // 32 columns inside [largest lim_lo, smallest lim) need no mask
                        const int hi_min = (int)__reduce_min_sync(0xffffffffu, (unsigned)min(max(lim, 0), 128));
                        const int lo_max = (int)__reduce_max_sync(0xffffffffu, (unsigned)min(max(lim_lo, 0), 128));
                        float *s = reinterpret_cast<float *>(&sr[0][0]);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if (32 * q >= lo_max && 32 * q + 32 <= hi_min) continue;
                            const uint32_t seen = (low_bits(lim - 32 * q) & ~low_bits(lim_lo - 32 * q)) |
                                                  low_bits(sk_hi - 32 * q) | (holds ? drafted[q] : 0u);
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(seen & (1u << c))) s[32 * q + c] = -INFINITY;
                        }
                    }
                };
                // P against the current reference, kept in registers until the
                // denominator has been checked; where it leaves its range the warp
                // reloads S, moves the reference to max(tile max, reference + log2 l),
                // rescales O, l and lr, and computes P again
                uint32_t pr[4][16];
                float lt, lrt;
                auto p_pass = [&]() {
                    const float *s = reinterpret_cast<const float *>(&sr[0][0]);
                    const uint64_t sl2x2 = f32x2(sl2, sl2), negm2 = f32x2(-m_ref, -m_ref);
                    uint64_t lsum[4] = {0ull, 0ull, 0ull, 0ull};
                    float rs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
#pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            float x0, x1;
                            f32x2_split(fma_f32x2(f32x2(s[32 * q + c], s[32 * q + c + 1]), sl2x2, negm2), x0, x1);
                            const float p0 = ex2(x0), p1 = ex2(x1);
                            lsum[(c >> 1) & 3] = add_f32x2(lsum[(c >> 1) & 3], f32x2(p0, p1));
                            const uint32_t pk = pack_bf16x2(p0, p1);
                            pr[q][c >> 1] = pk;
                            rs[(c >> 1) & 3] = add_bf16x2_to_f32(rs[(c >> 1) & 3], pk);
                        }
                    }
                    float a0, a1, b0, b1, c0, c1, d0, d1;
                    f32x2_split(lsum[0], a0, a1);
                    f32x2_split(lsum[1], b0, b1);
                    f32x2_split(lsum[2], c0, c1);
                    f32x2_split(lsum[3], d0, d1);
                    lt = ((a0 + a1) + (b0 + b1)) + ((c0 + c1) + (d0 + d1));
                    lrt = (rs[0] + rs[1]) + (rs[2] + rs[3]);
                };
                load_s();
                p_pass();
                {
                    const float ln = l + lt;
                    // (a row may see no column of a tile that its unit visits)
                    const bool bad = !(ln >= kTreeSumLo && ln <= kTreeSumHi) && live &&
                                     (max(lim_lo, 0) < min(lim, 128) || sk_hi > 0 || any_drafted);
                    if (__builtin_expect(__any_sync(0xffffffffu, bad), 0)) {
                        load_s();
                        const float *s = reinterpret_cast<const float *>(&sr[0][0]);
                        float mA = s[0], mB = s[1];
#pragma unroll
                        for (int c = 2; c < 126; c += 4) {
                            mA = max3(mA, s[c], s[c + 1]);
                            mB = max3(mB, s[c + 2], s[c + 3]);
                        }
                        mA = max3(mA, s[126], s[127]);
                        float m_new = m_ref;
                        if (bad) {
                            const float cand = fmaxf(fmaxf(mA, mB) * sl2, l > 0.f ? m_ref + lg2(l) : -INFINITY);
                            if (cand != -INFINITY) m_new = cand;
                        }
                        const float alpha = l > 0.f ? ex2(m_ref - m_new) : 1.f;
                        l *= alpha;
                        lr *= alpha;
                        m_ref = m_new;
                        if (mine > 0) {
                            if (!(ok = warp_wait(BAR(B_PVDONE + g), (n - 1) & 1, abort_flag))) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int q = 0; q < D / 16; ++q) {
                                uint32_t o[16];
                                tmem_ld16(tO + q * 16, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                                tmem_st16(tO + q * 16, o);
                            }
                            tmem_wait_st();
                        }
                        p_pass();
                    }
                }
                l += lt;
                lr += lrt;
                tc_fence_before();
                mbar_arrive(BAR(B_SFREE + g));
                j += step;
                first_new -= 128 * step;
                if (sq.window > 0) first_new = tree_tile(e, j) * 128 - e.before;    // (the sinks' tiles)
                // P_g's place is free once the product before has read it, and a segment's first
                // product may write O once both groups have read the last one's
                if (!settle()) break;
                if (mine > 0 && !(ok = warp_wait(BAR(B_PVDONE + g), (n - 1) & 1, abort_flag))) break;
                if constexpr (P_IN_TMEM) {
                    const uint32_t tP = tmem + lane_off + 384 + g * 64;
                    tmem_st32(tP, *reinterpret_cast<const uint32_t(*)[32]>(&pr[0][0]));
                    tmem_st32(tP + 32, *reinterpret_cast<const uint32_t(*)[32]>(&pr[2][0]));
                    tmem_wait_st();
                    tc_fence_before();
                } else {
                    uint32_t xr = (uint32_t)(r & 7) << 4;
                    asm volatile("" : "+r"(xr));
                    const uint32_t prow = s_base + L::kP + g * 2 * L::kBox + (r >> 3) * 1024 + xr * 8;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const uint32_t off = (q >> 1) * L::kBox + ((((q & 1) * 4 + m) << 4) ^ xr);
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(prow + off),
                                         "r"(pr[q][4 * m]), "r"(pr[q][4 * m + 1]), "r"(pr[q][4 * m + 2]),
                                         "r"(pr[q][4 * m + 3])
                                         : "memory");
                        }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                mbar_arrive(BAR(B_PFULL + g));
                ++mine;
                ++n;
            }
            let_go();
            if (!ok) break;
            // ---- the rows go out: final ones, or to the workspace, as a piece or a segment's parts so far
            // (a sum that is NaN keeps its reference, so that what it is added to becomes NaN too)
            float m_out = l == 0.f ? -INFINITY : m_ref;
            const size_t tok = (size_t)e.t0 + my_tok;
            const int head = e.hk * sq.group + my_head, tiles = e.tiles;
            const size_t to = (tok * sq.H + head) * D;
            bool final = e.whole != 0;
            if constexpr (PARTS) final = final && e.left == 0;
            const bool stored = live;
            const size_t slot = ((size_t)blockIdx.x * 2 + (e.begins ? 1 : 0)) * 2;
            // the next segment is made ready while the last products run
            more = begin(seg + 1);
            if (ok && mine > 0) {
                ok = warp_wait(BAR(B_PVDONE + g), (n - 1) & 1, abort_flag);
                tc_fence_after();
            }
            if (!ok) break;
            float4 *part_o = args.part_o + slot * (D / 4) * 128 + r, *part_ml = args.part_ml + slot * 128 + r;
            if constexpr (PARTS) {
                if (e.earlier != 0 && warp_live && (two || g == 0)) {
                    // the parts before are added to this one's O.  (Where the groups share the rows, each
                    // wrote half of the columns; they have met since.)
                    const float4 before = part_ml[g * 128];
                    const float top = fmaxf(m_out, before.x);
                    const float mine_f = m_out > -INFINITY ? ex2(m_out - top) : 0.f;
                    const float before_f = before.x > -INFINITY ? ex2(before.x - top) : 0.f;
                    m_out = top;
                    l = l * mine_f + before.y * before_f;
                    lr = lr * mine_f + before.z * before_f;
#pragma unroll 1
                    for (int q = 0; q < D / 16; ++q) {
                        uint32_t o[16];
                        tmem_ld16(tO + q * 16, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 16; c += 4) {
                            const float4 y = part_o[((two ? g * (D / 4) : 0) + 4 * q + c / 4) * 128];
                            o[c] = __float_as_uint(__uint_as_float(o[c]) * mine_f + y.x * before_f);
                            o[c + 1] = __float_as_uint(__uint_as_float(o[c + 1]) * mine_f + y.y * before_f);
                            o[c + 2] = __float_as_uint(__uint_as_float(o[c + 2]) * mine_f + y.z * before_f);
                            o[c + 3] = __float_as_uint(__uint_as_float(o[c + 3]) * mine_f + y.w * before_f);
                        }
                        tmem_st16(tO + q * 16, o);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
            }
            auto rows16 = [&](int gg, int q, bool there, float (&x)[16]) {     // columns 16 q .. of group gg's O
                uint32_t o[16];
                if (there) {
                    tmem_ld16(tO + (gg - g) * D + q * 16, o);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int c = 0; c < 16; ++c) x[c] = there ? __uint_as_float(o[c]) : 0.f;
            };
            auto put16 = [&](int q, const float (&x)[16], float inv) {
#pragma unroll
                for (int c = 0; c < 16; c += 8) {
                    const float y[8] = {x[c], x[c + 1], x[c + 2], x[c + 3], x[c + 4], x[c + 5], x[c + 6], x[c + 7]};
                    if (final) {
                        tree_store8(args, to, 16 * q + c, y, inv);
                    } else {
                        float4 *dst = part_o + ((two ? g * (D / 4) : 0) + 4 * q + c / 4) * 128;
                        dst[0] = make_float4(y[0], y[1], y[2], y[3]);
                        dst[128] = make_float4(y[4], y[5], y[6], y[7]);
                    }
                }
            };
            if (two || tiles == 0) {
                if (warp_live && (g == 0 || two)) {
                    const float inv = lr > 0.f ? 1.f / lr : 0.f;
#pragma unroll 2
                    for (int q = 0; q < D / 16; ++q) {
                        float x[16];
                        rows16(g, q, mine > 0, x);
                        if (stored) put16(q, x, inv);
                    }
                    if (!final) part_ml[g * 128] = make_float4(m_out, l, lr, 0.f);
                    else if (stored) tree_store_lse(args, tok, head, m_out, l);
                }
            } else {
                // both groups have the same rows: each adds half of the columns of both (a
                // warp reaches its lanes of all tensor memory)
                const uint32_t sums = s_base + L::kP + r * 16;   // group g's at 2 g boxes, where its P was read
                if (!settle()) break;
                st_shared_f4(sums + g * 2 * L::kBox, make_float4(m_out, l, lr, 0.f));
                arrive();
                if (!settle()) break;
                if (warp_live) {
                    tc_fence_after();
                    const float4 other = ld_shared_f4(sums + (1 - g) * 2 * L::kBox);
                    const float top = fmaxf(m_out, other.x);
                    const float mine_f = m_out > -INFINITY ? ex2(m_out - top) : 0.f;
                    const float other_f = other.x > -INFINITY ? ex2(other.x - top) : 0.f;
                    const float sum = lr * mine_f + other.z * other_f, inv = sum > 0.f ? 1.f / sum : 0.f;
                    const bool theirs = tiles > 1 || g == 1;       // (group 1 may have taken no tile)
#pragma unroll 1
                    for (int q = g * (D / 32); q < (g + 1) * (D / 32); ++q) {
                        float x[16], y[16];
                        rows16(g, q, mine > 0, x);
                        rows16(1 - g, q, theirs, y);
#pragma unroll
                        for (int c = 0; c < 16; ++c) x[c] = x[c] * mine_f + y[c] * other_f;
                        if (stored) put16(q, x, inv);
                    }
                    if (g == 0) {
                        const float both = l * mine_f + other.y * other_f;
                        if (!final) part_ml[0] = make_float4(top, both, sum, 0.f);
                        else if (stored) tree_store_lse(args, tok, head, top, both);
                    }
                    tc_fence_before();
                }
                arrive();            // (waited for before either group's O is written anew)
            }
            tc_fence_before();       // the next segment's first product may overwrite O
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(B_SEGFREE + (seg & 1)));
        }
        if (!ok) timed_out();
    }

    // ---- teardown: every role is here, all tensor-core work has finished
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The main kernel for units that may be longer than kTreePart tiles (attn_paged_tree_long.cu).
using TreeKernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, TreeArgs);
TreeKernel tree_kernel_in_parts(int d, bool two);

// The rows of cut units from their pieces, in their order: m = max m_i, l = sum l_i
// 2^(m_i - m), O = sum O_i 2^(m_i - m) / lr.  The blocks find the units that are cut in the
// CTAs' notes and share them, `slices` to a unit; eight columns of a row to a
// thread, AHEAD pieces on their way at once: ten where few units are cut into many,
// three and more blocks to an SM where many are cut into few.  Bound by latency:
// notes, pieces, rows.
template <int D, int AHEAD>
__global__ void __launch_bounds__(256, AHEAD > 4 ? 1 : 3) paged_tree_join_kernel(const __grid_constant__ TreeArgs a, int ctas) {
    __shared__ int found[8], of_mine;
    __shared__ TreeCut mine_cut;
    pdl_wait();
    static_assert(kTreeCtas <= 256, "a thread to each CTA's note");
    TreeCut cut{0, 0, 0, 0};
    if ((int)threadIdx.x < ctas) cut = a.cuts[threadIdx.x];
    const unsigned warp_cuts = __ballot_sync(0xffffffffu, cut.n > 0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) found[warp] = __popc(warp_cuts);
    __syncthreads();
    int units = 0, before = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        if (w < warp) before += found[w];
        units += found[w];
    }
    if (units == 0) return;
    const int slices = max((int)gridDim.x / units, 1), unit = blockIdx.x / slices, slice = blockIdx.x - unit * slices;
    if (unit >= units) return;
    if (cut.n > 0 && before + __popc(warp_cuts & ((1u << lane) - 1)) == unit) {
        mine_cut = cut;
        of_mine = threadIdx.x;
    }
    __syncthreads();
    cut = mine_cut;
    const int cta0 = of_mine, group = a.seqs.group, rows = cut.n * group, share = (rows + slices - 1) / slices;
    const int row0 = min(slice * share, rows), n = min(row0 + share, rows) - row0, pieces = cut.more + 1;
    for (int i = threadIdx.x; i < n * (D / 8); i += 256) {
        const int c8 = i / n, row = row0 + i - c8 * n, tok = row / group, head = cut.hk * group + row - tok * group;
        const int late = a.two && tok >= a.tile_tokens ? 1 : 0, r = row - late * a.tile_tokens * group;
        float x[8] = {}, top = -INFINITY, l = 0.f, lr = 0.f;
        for (int p0 = 0; p0 < pieces; p0 += AHEAD) {
            float4 f[AHEAD][2], m[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                const int p = min(p0 + j, pieces - 1);
                const size_t at = ((size_t)(cta0 + p * a.streams) * 2 + (p == 0 ? 1 : 0)) * 2 + late;
                const float4 *o = a.part_o + (at * (D / 4) + 2 * c8) * 128 + r;
                m[j] = a.part_ml[at * 128 + r];
                f[j][0] = o[0];
                f[j][1] = o[128];
                if (p0 + j >= pieces) m[j].x = -INFINITY;
            }
            float t2 = top;
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) t2 = fmaxf(t2, m[j].x);
            if (!(t2 > -INFINITY)) continue;
            const float old = ex2(top - t2);
#pragma unroll
            for (int c = 0; c < 8; ++c) x[c] *= old;
            l *= old;
            lr *= old;
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                if (!(m[j].x > -INFINITY)) continue;
                const float now = ex2(m[j].x - t2);
                const float4 y = f[j][0], z = f[j][1];
                x[0] += y.x * now, x[1] += y.y * now, x[2] += y.z * now, x[3] += y.w * now;
                x[4] += z.x * now, x[5] += z.y * now, x[6] += z.z * now, x[7] += z.w * now;
                l += m[j].y * now;
                lr += m[j].z * now;
            }
            top = t2;
        }
        const size_t t = (size_t)cut.t0 + tok;
        tree_store8(a, (t * a.seqs.H + head) * D, 8 * c8, x, lr > 0.f ? 1.f / lr : 0.f);
        if (c8 == 0) tree_store_lse(a, t, head, top, l);
    }
}

}  // namespace ra
