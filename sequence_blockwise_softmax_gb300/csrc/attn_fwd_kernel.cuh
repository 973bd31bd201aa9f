// attn_fwd_kernel.cuh -- blockwise exact attention on the sm_103a tensor cores.
//
// One CTA owns a "unit": 256 query rows (two 128-row Q tiles) of one
// (query rank, batch, head).  It sweeps the key/value shards in ring order
// ("From Ring Attention to DeepSpeed Ulysses to USP", jsqmd.com/news/734632,
// §3.1: at step s rank i holds the KV of rank (i - s) mod N) and folds every
// 128-key tile into the running (m, l, O) state of §3.2, so the partial
// results never leave the SM.  Here m is the reference point of the
// exponentials, not necessarily the running max (see kSumLo below).
//
// Causal masking by position (same article §3.4; "What problem does sequence
// parallelism solve?", model.playoffer.cn, engineering notes: the ring decides
// the mask from the token positions).  In every layout a rank's local tokens
// are in increasing global order, so the keys of shard j that query row a may
// see are exactly a prefix 0..kc(a)-1 of that shard.  A unit visits only the
// key tiles that prefix covers for its last row (fully masked tiles are
// skipped), and each softmax thread masks the columns past its own row's
// prefix (diagonal tiles are masked in-tile).
//
// Warp roles (384 threads):
//   warp 0      TMA producer: Q tiles once, then K and V tiles into one ring
//               of three shared-memory slots, K a tile ahead of V.
//   warp 1      MMA issuer (one elected lane): S_g = Q_g K^T into tensor
//               memory, and at d = 64 also O_g += P_g V with P_g read from
//               tensor memory.
//   warp 2      tensor-memory allocator.
//   warp 3      at d = 128, the PV issuer, so that a wait of either issuer
//               never holds back the other's products (the tensor pipe takes
//               only a few MMAs ahead of execution).
//   warps 4-7   softmax for Q tile 0, warps 8-11 for Q tile 1: one thread per
//               query row (the 32x32b tensor-memory load gives a thread its
//               whole row, so row sums need no shuffles), exp2 with the
//               scale folded into log2(e), P written as bf16 to shared memory
//               (d = 128) or tensor memory (d = 64), O rescaled in place when
//               the reference point moves,
//               and the final normalisation, with O staged in shared memory
//               for TMA stores.  At d = 128 warp 4 first counts the unit's
//               key tiles for the two issuers, one ring step per lane.
// Tensor memory (512 columns x 128 lanes): S_0 [0,128), S_1 [128,256),
// O_0 [256, 256+d), O_1 [256+d, 256+2d), and at d = 64 P_0 [384, 448),
// P_1 [448, 512) (bf16 pairs), which PV reads from there; at d = 128 P goes
// through shared memory.  Because P does not live in S's
// columns, S_g(t+1) may be computed while PV_g(t) still runs: the softmax
// releases S_g once P is computed and its denominator checked (the rare
// second pass reloads S), and each tile's critical chain is S -> softmax ->
// PV with no wait on the previous PV in between.
//
// Addressing: every tile moves through a 4-D tensor map of either the shard
// stacks [N, B, S, H, d] or the token-order tensors [B, L, H, d]
// (tile_view / tile_coords).  In token order a layout is only a choice of view
// (§4, §6.1 of the same article), so the sweep reads each rank's shard and
// writes its result in place and no permute runs.
#pragma once
#include <type_traits>

#include "kv_tile.cuh"
#include "ra_device.cuh"
#include "ra_internal.h"
#include "ra_paged.cuh"
#include "ra_positions.cuh"
#include "ra_window.cuh"

namespace ra {

struct AttnArgs {
    void *o;
    float *lse;
    unsigned *status;
    int B, S, H, N;
    int layout, causal;
    float scale_log2;   // softmax scale * log2(e)
    int num_q_ranks;    // N in ring mode, 1 in block mode
    int q_rank_fixed;   // block mode: the query rank; ring mode: -1
    int kv_rank_fixed;  // block mode: the key/value rank; ring mode: -1
    int num_steps;      // N for a full sweep, 1 for one ring step or block mode
    int step_base;      // ring mode: the first step visited (0 for a full sweep)
    int n_units_seq;    // ceil(S / 256)
    int inject_stall;   // test hook: CTA 0 never loads its second K tile
    int kv_group;       // query heads per key/value head (1 without GQA)
    const int *cu_seqlens;  // packed sequences: n_seqs + 1 boundaries, or null
    int n_seqs;
    int bh_chunk;       // (batch, head) pairs whose units are interleaved heavy-first
    int seq_order;      // q/k/v/o in sequence order [B, L, H, d], LSE [B, H, L] (ring mode)
    int window, sinks;  // windowed keys (KEYS_WINDOW)
    int whole_units;    // and its units of 256 rows; the others run in halves
    // KEYS_PAGED: the sequences and pages; the parts' rows when the keys are
    // split, [units, H_kv, num_splits, rows of a unit, d], and their LSE
    PagedSeqs seqs;
    int n_units, tile_tokens, page_box, o_bf16;
    float *part_o, *part_lse;
};

// Which keys a unit's rows see.  KEYS_RING: the shards of a ring sweep, by
// position.  KEYS_WINDOW: one batch element's own tokens (N = 1), a causal
// window and the sequence's first tokens (window_row_keys).  KEYS_PAGED: new
// tokens over a paged cache (ra_paged.cuh): a unit's rows are the group of
// query heads of up to 2 * tile_tokens tokens, its key tiles are gathered from
// the block table's pages, and its tiles may be split over several CTAs.
enum KeySet { KEYS_RING = 0, KEYS_WINDOW = 1, KEYS_PAGED = 2 };

// The sequence of unit u, searched by a whole warp: 32 probes at a time.
__device__ __forceinline__ int paged_find_seq_warp(const PagedSeqs &q, int u, int lane) {
    int lo = 0, hi = q.n_seqs;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const bool below = at < hi && (lane == 0 || paged_first_unit(q, at) <= u);
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, below));
        lo += last * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// The at-th unit of a call with up to 32 sequences, the longest sequence's last
// unit first (its number in its sequence, or -1 past the last one); the whole
// warp gets the same answer.  Long units that start last leave SMs idle.
__device__ __forceinline__ int paged_sorted_unit(const PagedSeqs &q, int n_units, int at, int lane, int &seq) {
    int len = -1, units = 0;
    if (lane < q.n_seqs) {
        len = paged_len(q, lane);
        units = max((lane + 1 < q.n_seqs ? paged_first_unit(q, lane + 1) : n_units) - paged_first_unit(q, lane), 0);
    }
    int before = 0;       // units of longer sequences
    for (int j = 0; j < q.n_seqs; ++j) {
        const int other = __shfl_sync(0xffffffffu, len, j), n = __shfl_sync(0xffffffffu, units, j);
        if (other > len || (other == len && j < lane)) before += n;
    }
    const int local = units - 1 - (at - before);
    const unsigned mine = __ballot_sync(0xffffffffu, local >= 0 && local < units);
    seq = mine ? __ffs(mine) - 1 : 0;
    return mine ? __shfl_sync(0xffffffffu, local, seq) : -1;
}

__device__ __forceinline__ void record_timeout(unsigned *status, volatile int *abort) {
    *abort = 1;
    atomicOr(status, RA_DEV_TIMEOUT_BIT);
}

template <int D>
struct AttnSmem {
    static constexpr int kSlots = 3;                     // K/V tile ring
    static constexpr uint32_t kTile = 128u * D * 2u;     // 128 rows x d bf16
    static constexpr uint32_t kBox = 128u * 128u;        // 128 rows x 64 columns
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kRing = 2 * kTile;
    static constexpr uint32_t kP = kRing + kSlots * kTile;   // P_g: 128 rows x 128 keys bf16, two boxes each
    static constexpr uint32_t kBars = kP + 2 * 2 * kBox;
    // barriers: Q full, K full[3], V full[3], slot empty[3], S full[2],
    // S free[2], P full[2], PV done[2], final, tile count posted.  A slot holds
    // K and V loads in turn but has a full barrier for each: the S and the PV
    // issuer then see every phase of the barriers they wait on.  On one shared
    // barrier each would see every other phase, and a wait two phases ahead of
    // the barrier passes at once (the parities agree): products would read a
    // tile still on its way whenever loads lag or overtake one another.
    static constexpr int kNumBars = 1 + 3 * kSlots + 2 + 2 + 2 + 2 + 1 + 1;
    static constexpr uint32_t kMisc = kBars + kNumBars * 8;
    // the tile-skipping variant's step table: per ring step (at most
    // kMaxSteps) the unit's key-tile range and each Q tile's own range inside
    // it, six ints
    static constexpr int kMaxSteps = 64;
    static constexpr uint32_t kTab = kMisc + 16;
    // no alignment slack: the kernel requires (and checks) a 1024-byte-aligned
    // dynamic base, which is what leaves room for P
    static constexpr uint32_t kBytes = kMisc + 16;
    static constexpr uint32_t kBytesSkip = kTab + kMaxSteps * 6 * 4;
};

// The key tiles of a unit's walk as the tile-skipping variant sees them: the
// walk visits tiles [lo, hi) of each step's shard in step order, and Q tile g
// needs only tiles [glo_g, ghi_g) of them.  With no table (more steps than it
// holds) every tile is needed by both Q tiles.
struct StepCursor {
    const int *tab;   // null: no table
    int ns, s, tile, hi, lo0, hi0, lo1, hi1;   // the current step's ranges
    __device__ void seek() {
        while (s < ns && tab[6 * s] >= tab[6 * s + 1]) ++s;
        if (s < ns) {
            tile = tab[6 * s];
            hi = tab[6 * s + 1];
            lo0 = tab[6 * s + 2];
            hi0 = tab[6 * s + 3];
            lo1 = tab[6 * s + 4];
            hi1 = tab[6 * s + 5];
        }
    }
    __device__ void start(const int *t, int n) {
        tab = t;
        ns = n;
        s = 0;
        tile = 0;
        if (tab) seek();
    }
    __device__ void next() {
        if (tab && ++tile >= hi) {
            ++s;
            seek();
        }
    }
    __device__ bool need(int g) const {
        return !tab || (g == 0 ? (lo0 <= tile && tile < hi0) : (lo1 <= tile && tile < hi1));
    }
};

// Reference point of the exponentials.  The online softmax of §3.2 subtracts
// the running row max m only to keep exp() in range: O / l and m + ln l are
// the same for any reference.  A row therefore starts at reference 0 and
// computes P = 2^(s*scale*log2e - m) without a row max; the reference moves
// only when the running denominator would leave [kSumLo, kSumHi] (or is not
// a number), to max(tile max, m + log2 l), which brings the sum into
// [1, 129].  With l <= 2^32 no P and no partial sum of P can overflow, and
// with l >= 2^-32 over at most 2^24 keys the largest term is at least
// 2^-56, so what ex2 flushes to zero (below 2^-126) is less than 2^-70 of
// it.  For scores of ordinary size (|s * scale| up to about 20) the
// reference never moves at all.
constexpr float kSumLo = 0x1p-32f, kSumHi = 0x1p32f;

// SKIP: each Q tile of a unit skips the key tiles none of its own rows sees
// (packed sequences in the striped layout, where a unit's 256 rows span many
// short sequences); the MMA issuers skip those tiles' S and PV.
template <int D, bool OUT_F32, bool SKIP, int KEYS = KEYS_RING>
__global__ void __launch_bounds__(384, 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                    const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmo,
                    const AttnArgs args) {
    using L = AttnSmem<D>;
    constexpr int NSL = L::kSlots;
    constexpr int HALVES = D / 64;
    constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 128, false);
    constexpr uint32_t IDESC_O = idesc_bf16_f32(128, D, true);
    // At d = 128 warp 1 issues the S products and warp 3 the PV products; at
    // d = 64, where the split measured slower, warp 1 issues both.
    constexpr bool TWO_ISSUERS = D == 128;
    // At d = 64 tensor memory has room for P next to S and O (columns 384-511),
    // so P_g goes there and PV_g reads it as the A operand (a TS product): no
    // P stores through shared memory and no proxy fence.  At d = 128 S and O
    // fill all 512 columns and P goes through shared memory.
    constexpr bool P_IN_TMEM = D == 64;
    // registers per thread of warps 0-3 after setmaxnreg: the second issuer
    // needs more than 64 to issue without spilling
    constexpr uint32_t LOW_REGS = TWO_ISSUERS ? 72u : 64u;
    static_assert(!SKIP || TWO_ISSUERS, "tile skipping is built on the two-issuer pipeline");
    static_assert(!SKIP || KEYS == KEYS_RING, "tile skipping is a variant of the ring sweep");
    using Walk = typename std::conditional<KEYS == KEYS_RING, TileWalk, RangeWalk>::type;
    using KT = KvTile<D, KEYS == KEYS_PAGED && D == 128>;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    if constexpr (KEYS != KEYS_RING) pdl_wait();   // launched with launch_dependent()
    uint8_t *smem = smem_raw;
    const uint32_t s_base = smem_u32(smem);
    if ((s_base & 1023u) != 0u) {
        if (threadIdx.x == 0) atomicOr(args.status, RA_DEV_SMEM_ALIGN_BIT);
        return;
    }
    const uint32_t bar0 = s_base + L::kBars;
    auto BAR = [&](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
    const int B_QFULL = 0, B_KF = 1, B_VF = 1 + NSL, B_SLOTE = 1 + 2 * NSL, B_SFULL = 1 + 3 * NSL, B_SFREE = B_SFULL + 2,
              B_PFULL = B_SFREE + 2, B_PVDONE = B_PFULL + 2, B_FINAL = B_PVDONE + 2, B_TCOUNT = B_FINAL + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);
    volatile int *tile_count = reinterpret_cast<volatile int *>(smem + L::kMisc + 8);
    volatile int *tab_ok = reinterpret_cast<volatile int *>(smem + L::kMisc + 12);
    int *step_tab = reinterpret_cast<int *>(smem + L::kTab);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    // ---- unit decode: heavy units first, in L2-sized chunks of (batch, head)
    // pairs (decode_unit)
    const int H = args.H, N = args.N;
    // KEYS_WINDOW: the tokens in sequences; rows behind them are left alone
    const int S = KEYS == KEYS_WINDOW ? packed_tokens(args.cu_seqlens, args.n_seqs, args.S) : args.S;
    UnitId unit{};
    PagedUnit pu{};
    int part = 0;             // KEYS_PAGED: which part of the unit's keys
    bool split = false;       // ... and whether there is more than one
    int unit_no = 0;
    if constexpr (KEYS == KEYS_PAGED) {
        // Shorter last parts at the end.  Several sequences: blockIdx.x = (part *
        // n_units + at) * H_kv + hk, longer sequences and their last (longest)
        // units first.  One, or too many to sort here: (part * H_kv + hk) *
        // n_units + at, so that the CTAs of one head and part stand together and
        // share its keys in L2.
        int sq, local;
        if (args.seqs.n_seqs > 1 && args.seqs.n_seqs <= 32) {
            unit.h = blockIdx.x % args.seqs.Hkv;      // the key/value head
            const int rest = blockIdx.x / args.seqs.Hkv;
            part = rest / args.n_units;
            local = paged_sorted_unit(args.seqs, args.n_units, rest % args.n_units, lane, sq);
            if (local < 0) return;
            unit_no = paged_first_unit(args.seqs, sq) + local;
        } else {
            const int rest = blockIdx.x / args.n_units;
            unit.h = rest % args.seqs.Hkv;
            part = rest / args.seqs.Hkv;
            unit_no = args.n_units - 1 - blockIdx.x % args.n_units;
            sq = paged_find_seq_warp(args.seqs, unit_no, lane);
            local = unit_no - paged_first_unit(args.seqs, sq);
        }
        pu = paged_unit(args.seqs, sq, local);
        if (part == 0 && unit.h == 0 && threadIdx.x == 0 && pu.first == 0 && paged_bad_counts(args.seqs, sq))
            atomicOr(args.status, RA_DEV_PAGE_BIT);
        if (pu.n <= 0) return;
    } else {
        unit = decode_unit(KEYS == KEYS_WINDOW ? window_rows(blockIdx.x, args.whole_units).unit : (int)blockIdx.x,
                           args.bh_chunk, args.B, H, args.num_q_ranks, args.n_units_seq, args.layout);
    }
    const int b = unit.b, h = unit.h, qi = unit.qi, qt = unit.qt;
    const bool ring = args.q_rank_fixed < 0;
    const int q_rank = ring ? qi : args.q_rank_fixed;
    const int zq = (ring ? qi * args.B : 0) + b;
    // (a half unit's other Q tile sees no key and is not stored)
    const WindowRows wr = KEYS == KEYS_WINDOW ? window_rows(blockIdx.x, args.whole_units) : WindowRows{0, -1};
    const int row0 = wr.first(qt * 256);
    if (KEYS == KEYS_WINDOW && row0 >= S) return;
    const int row_end = min(S, row0 + wr.rows());
    // first row of a key tile that is to be read as zeros (KEYS_PAGED: behind the
    // sequence; KEYS_WINDOW: behind the last one; past args.S the copy gives zeros)
    auto zeros_from = [&](int tile) -> int {
        if (KEYS == KEYS_PAGED) return pu.len - tile * 128;
        return KEYS == KEYS_WINDOW && S < args.S ? S - tile * 128 : 128;
    };

    Walk walk0;
    if constexpr (KEYS == KEYS_RING)
        walk0 = unit_walk(args.layout, N, S, q_rank, args.kv_rank_fixed, args.num_steps, args.step_base, row0,
                          row_end, args.causal, args.cu_seqlens, args.n_seqs);
    else if constexpr (KEYS == KEYS_WINDOW)
        walk0 = window_unit_walk(args.cu_seqlens, args.n_seqs, S, row0, row_end, args.window, args.sinks);
    else {
        walk0 = paged_walk(args.seqs, pu);
        if (args.seqs.num_splits > 1) {
            const int parts = paged_split_count(args.seqs, walk0.end);
            if (part >= parts) return;
            split = parts > 1;
            const int per = paged_split_tiles(args.seqs, walk0.end);
            walk0.i = part * per;
            walk0.end = min(walk0.end, walk0.i + per);
        }
    }
    // KEYS_PAGED: a unit of few tokens has no second Q tile; its products and
    // softmax are left out
    const bool two_tiles = KEYS != KEYS_PAGED || pu.n > args.tile_tokens;
    // KEYS_WINDOW: a Q tile's products and softmax skip the key tiles that only
    // the other one's rows see (its neighbour's diagonal, its window's start):
    // one of 9 and more at a window of 1024, one of 4 at 128
    constexpr bool EDGES = KEYS == KEYS_WINDOW;
    auto w_tile = [](const auto &w) -> int { return w.tile; };
    auto seen_by = [&](int g) -> SeenTiles {
        const int fr = row0 + 128 * g;
        if (!EDGES || fr >= row_end) return SeenTiles{0, 0, 0, 0};
        return seen_tiles(window_row(args.cu_seqlens, args.n_seqs, S, fr, args.window, args.sinks),
                          min(row_end, fr + 128));
    };

    // ---- setup
    if (threadIdx.x == 0) {
        mbar_init(BAR(B_QFULL), 1);
        for (int s = 0; s < NSL; ++s) {
            mbar_init(BAR(B_KF + s), 1);
            mbar_init(BAR(B_VF + s), 1);
            mbar_init(BAR(B_SLOTE + s), 1);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(BAR(B_SFULL + g), 1);
            mbar_init(BAR(B_SFREE + g), 128);
            mbar_init(BAR(B_PFULL + g), 128);
            mbar_init(BAR(B_PVDONE + g), 1);
        }
        mbar_init(BAR(B_FINAL), TWO_ISSUERS ? 2 : 1);   // one arrival per MMA issuer
        mbar_init(BAR(B_TCOUNT), 1);
        *abort_flag = 0;
        fence_mbar_init();
        if constexpr (KEYS == KEYS_WINDOW) {
            // Q and K(0) are on their way before tensor memory is allocated and
            // the roles start: short units live by their prologue
            mbar_arrive_expect_tx(BAR(B_QFULL), 2 * L::kTile);
            for (int g = 0; g < 2; ++g)
                for (int c = 0; c < HALVES; ++c)
                    tma_load_4d(s_base + L::kQ + g * L::kTile + c * L::kBox, &tmq, BAR(B_QFULL), h * D + 64 * c,
                                row0 + 128 * g, b, 0);
            if (walk0.valid()) {
                Walk w0 = walk0;
                w0.start_step();
                mbar_arrive_expect_tx(BAR(B_KF), L::kTile);
                for (int c = 0; c < HALVES; ++c)
                    tma_load_4d(s_base + L::kRing + c * L::kBox, &tmk, BAR(B_KF), (h / args.kv_group) * D + 64 * c,
                                w0.tile * 128, b, 0);
            }
        }
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
        tma_prefetch_desc(&tmo);
    }
    if (warp == 2) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // 384 threads x 168 registers at launch: the producer / MMA / allocator
    // warpgroup (warps 0-3) gives registers to the two softmax warpgroups,
    // 128 x LOW_REGS + 256 x 216 <= 384 x 168 (equal at LOW_REGS = 72); each
    // role makes the call on entry.
    if (warp == 0) {
        // ================================================= TMA producer
        regs_shrink<LOW_REGS>();
        const int xh = h * D;                        // Q columns of head h
        const int xkv = KEYS == KEYS_PAGED ? h * D : (h / args.kv_group) * D;   // K/V columns of its key/value head
        if constexpr (KEYS == KEYS_PAGED) {
            // a box of the group's heads by tile_tokens tokens: rows in the
            // packed order; rows of later tokens of q are loaded but not used
            if (lane == 0) {
                const int tiles = two_tiles ? 2 : 1;
                mbar_arrive_expect_tx(BAR(B_QFULL), tiles * HALVES * args.tile_tokens * args.seqs.group * 128);
                for (int g = 0; g < tiles; ++g)
                    for (int c = 0; c < HALVES; ++c)
                        tma_load_3d(s_base + L::kQ + g * L::kTile + c * L::kBox, &tmq, BAR(B_QFULL), 64 * c,
                                    h * args.seqs.group, pu.t0 + g * args.tile_tokens);
            }
        } else if (KEYS == KEYS_RING && lane == 0) {
            mbar_arrive_expect_tx(BAR(B_QFULL), 2 * L::kTile);
            for (int g = 0; g < 2; ++g) {
                int c1, c2, c3;
                tile_coords(args.seq_order, args.layout, args.S, args.N, ring ? qi : 0, b, row0 + 128 * g, c1, c2, c3);
                for (int c = 0; c < HALVES; ++c)
                    tma_load_4d(s_base + L::kQ + g * L::kTile + c * L::kBox, &tmq, BAR(B_QFULL),
                                xh + 64 * c, c1, c2, c3);
            }
        }
        __syncwarp();
        // K and V tiles share a ring of three slots.  Load order K(0), K(1),
        // V(0), K(2), V(1), ...: K runs a tile ahead, because S(t+1) is issued
        // while P(t) is still being built.  Load i goes to slot i % 3 once the
        // load three before it has been released (K after both S products of
        // its tile, V after both PV products).
        // one walk over the key tiles; V(t) reuses the coordinates K(t) had
        Walk wk = walk0;
        wk.start_step();
        int vj = 0, vtile = 0;
        int i = 0, withheld = -1;
        uint32_t k_loads = 0, v_loads = 0;   // bit s: slot s has had a load of the kind, bit 8 + s: the parity of its last
        bool ok = true;
        // KEYS_PAGED: lane i's page of a key tile (its box of page_box keys), or
        // one past the last page, which reads as zeros, where the unit sees none
        // of its keys
        const RowKeys first = KEYS == KEYS_PAGED ? paged_row(args.seqs, pu.p0) : RowKeys{};
        auto page_of = [&](int wtile) -> int {
            int z = args.seqs.n_pages;
            const int k0 = wtile * 128 + lane * args.page_box;
            if (lane * args.page_box < 128 && paged_needed(first, pu.p0 + pu.n, pu.len, k0, args.page_box)) {
                z = args.seqs.table[(size_t)pu.s * args.seqs.max_pages + k0 / args.seqs.page];
                if ((unsigned)z >= (unsigned)args.seqs.n_pages) {
                    atomicOr(args.status, RA_DEV_PAGE_BIT);
                    z = args.seqs.n_pages;
                }
            }
            return z;
        };
        // (for KEYS_PAGED wj is the lane's page)
        auto load = [&](int wj, int wtile, bool is_k) -> bool {
            const int sl = i % NSL;
            if (i >= NSL && !warp_wait(BAR(B_SLOTE + sl), ((i / NSL) - 1) & 1, abort_flag)) return false;
            const bool withhold = args.inject_stall && blockIdx.x == 0 && i == 1;
            const uint32_t full = BAR((is_k ? B_KF : B_VF) + sl);
            uint32_t &loads = is_k ? k_loads : v_loads;
            loads = (loads & (1u << sl)) ? loads ^ (256u << sl) : loads | (1u << sl);
            if constexpr (KEYS == KEYS_PAGED) {
                const uint32_t dst = s_base + L::kRing + sl * L::kTile;
                if (lane == 0) mbar_arrive_expect_tx(full, L::kTile);
                __syncwarp();
                if (lane * args.page_box < 128) {
                    const int y = (wtile * 128 + lane * args.page_box) & (args.seqs.page - 1);
                    const uint32_t to = dst + (lane * args.page_box >> 3) * KT::kGroup;
                    if constexpr (HALVES == 2)
                        tma_load_5d(to, is_k ? &tmk : &tmv, full, 0, 0, 2 * h, y >> 3, wj);
                    else
                        tma_load_3d(to, is_k ? &tmk : &tmv, full, xkv, y, wj);
                }
            } else if (lane == 0 && !withhold && !(KEYS == KEYS_WINDOW && i == 0)) {   // (K(0): issued in the setup)
                const uint32_t dst = s_base + L::kRing + sl * L::kTile;
                int c1, c2, c3;
                tile_coords(args.seq_order, args.layout, args.S, args.N, ring ? wj : 0, b, wtile * 128, c1, c2, c3);
                mbar_arrive_expect_tx(full, L::kTile);
                for (int c = 0; c < HALVES; ++c) {
                    if (is_k) tma_load_4d(dst + c * L::kBox, &tmk, full, xkv + 64 * c, c1, c2, c3);
                    else tma_load_4d(dst + c * L::kBox, &tmv, full, xkv + 64 * c, c1, c2, c3);
                }
            }
            __syncwarp();
            if (withhold) withheld = i;
            ++i;
            return true;
        };
        if constexpr (KEYS == KEYS_PAGED) {
            if (wk.valid()) wk.j = page_of(wk.tile);
            // the next tile's table entries are read a tile ahead
            while (ok && wk.valid()) {
                if (!(ok = load(wk.j, wk.tile, true))) break;
                if (i > 1 && !(ok = load(vj, vtile, false))) break;
                vj = wk.j;
                vtile = wk.tile;
                wk.next();
                if (wk.valid()) wk.j = page_of(wk.tile);
            }
            if (ok && i > 0) ok = load(vj, vtile, false);
        } else if (wk.valid()) {
            ok = load(wk.j, wk.tile, true);
            vj = wk.j;
            vtile = wk.tile;
            wk.next();
            while (ok) {
                const bool more = wk.valid();
                if (more && !(ok = load(wk.j, wk.tile, true))) break;
                if (!(ok = load(vj, vtile, false)) || !more) break;
                vj = wk.j;
                vtile = wk.tile;
                wk.next();
            }
        }
        if (!ok) {
            if (lane == 0) record_timeout(args.status, abort_flag);
            // let the copies already issued land before the CTA exits
            volatile int never = 0;
            mbar_wait(BAR(B_QFULL), 0, &never);
            for (int sl = 0; sl < NSL; ++sl) {
                if (((k_loads >> sl) & 1u) && !(withheld == 1 && sl == 1))   // (load 1 is a K tile)
                    mbar_wait(BAR(B_KF + sl), (k_loads >> (8 + sl)) & 1u, &never);
                if ((v_loads >> sl) & 1u) mbar_wait(BAR(B_VF + sl), (v_loads >> (8 + sl)) & 1u, &never);
            }
        }
    } else if (warp == 1 && !TWO_ISSUERS) {
        // ================================================= MMA issuer (d = 64)
        regs_shrink<LOW_REGS>();
        // Issue order per key tile t (pipe order):
        //   S_0(t+1), PV_0(t), S_1(t+1), PV_1(t)
        // P_g goes to shared memory, so S_g(t+1) may overwrite S_g(t) in
        // tensor memory as soon as the softmax warps of tile g are done with it
        // (S free); nothing here waits for a PV product.  Descriptors are built
        // once; each k-step adds a compile-time offset (16-byte units) to the
        // start-address field: 32 B per 16-element step inside a 64-column box
        // and one box (16 KB) for columns 64-127 of Q, K and P, and 16 rows
        // (2 KB) per step of V.  The whole warp runs the issue code and
        // elect.sync picks the issuing lane.
        const uint64_t dq[2] = {sdesc_sw128(s_base + L::kQ, 16, 1024),
                                sdesc_sw128(s_base + L::kQ + L::kTile, 16, 1024)};
        const uint64_t dp[2] = {sdesc_sw128(s_base + L::kP, 16, 1024),
                                sdesc_sw128(s_base + L::kP + 2 * L::kBox, 16, 1024)};
        const uint64_t dk0 = sdesc_sw128(s_base + L::kRing, 16, KT::kGroup);
        const uint64_t dv0 = sdesc_sw128(s_base + L::kRing, KT::kHalf, KT::kGroup);
        auto issue_s = [&](int g, int slot) {
            const uint64_t a0 = dq[g], b0 = dk0 + (uint64_t)(slot * (L::kTile >> 4));
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
        auto issue_pv = [&](int g, int slot, bool first) {
            constexpr uint32_t hb = L::kBox >> 4;
            const uint64_t a0 = dp[g], b0 = dv0 + (uint64_t)(slot * (L::kTile >> 4));
            const uint32_t d = tmem + 256 + g * D;
            if constexpr (P_IN_TMEM) {
                // A = P_g in tensor memory: 16 keys (8 packed columns) per k-step
                const uint32_t at = tmem + 384 + g * 64;
                mma_ts_elect<0, 0>(d, at, b0, IDESC_O, first ? 0u : 1u);
                mma_ts_elect<8, 128>(d, at, b0, IDESC_O, 1u);
                mma_ts_elect<16, 256>(d, at, b0, IDESC_O, 1u);
                mma_ts_elect<24, 384>(d, at, b0, IDESC_O, 1u);
                mma_ts_elect<32, 512>(d, at, b0, IDESC_O, 1u);
                mma_ts_elect<40, 640>(d, at, b0, IDESC_O, 1u);
                mma_ts_elect<48, 768>(d, at, b0, IDESC_O, 1u);
                mma_ts_elect<56, 896>(d, at, b0, IDESC_O, 1u);
            } else {
                mma_ss_elect<0, 0>(d, a0, b0, IDESC_O, first ? 0u : 1u);
                mma_ss_elect<2, 128>(d, a0, b0, IDESC_O, 1u);
                mma_ss_elect<4, 256>(d, a0, b0, IDESC_O, 1u);
                mma_ss_elect<6, 384>(d, a0, b0, IDESC_O, 1u);
                mma_ss_elect<hb, 512>(d, a0, b0, IDESC_O, 1u);
                mma_ss_elect<hb + 2, 640>(d, a0, b0, IDESC_O, 1u);
                mma_ss_elect<hb + 4, 768>(d, a0, b0, IDESC_O, 1u);
                mma_ss_elect<hb + 6, 896>(d, a0, b0, IDESC_O, 1u);
            }
            tc_commit_elect(BAR(B_PVDONE + g));
        };
        uint32_t k_parity = 0;   // bit s: parity of the next K load of slot s
        auto k_wait = [&](int sl) -> bool {
            const bool got = warp_wait(BAR(B_KF + sl), (k_parity >> sl) & 1u, abort_flag);
            k_parity ^= 1u << sl;
            return got;
        };
        uint32_t v_parity = 0;   // bit s: parity of the next V load of slot s
        auto v_wait = [&](int sl) -> bool {
            const bool got = warp_wait(BAR(B_VF + sl), (v_parity >> sl) & 1u, abort_flag);
            v_parity ^= 1u << sl;
            return got;
        };
        bool ok = warp_wait(BAR(B_QFULL), 0, abort_flag);
        Walk w = walk0;
        w.start_step();
        const SeenTiles seen0 = seen_by(0), seen1 = seen_by(1);
        auto need = [&](int g, int tile) -> bool {
            if (EDGES) return g == 0 ? seen0.has(tile) : seen1.has(tile);
            return g == 0 || two_tiles;
        };
        int n_s0 = 0, n_s1 = 0, n_p0 = 0, n_p1 = 0;   // products issued per Q tile
        int t = 0;
        if (ok && w.valid()) {
            ok = k_wait(0);   // K(0) is load 0
            tc_fence_after();
            if (ok) {
                if (need(0, w.tile)) {
                    issue_s(0, 0);
                    ++n_s0;
                }
                if (need(1, w.tile)) {
                    issue_s(1, 0);
                    ++n_s1;
                }
                tc_commit_elect(BAR(B_SLOTE + 0));
            }
            __syncwarp();
        }
        while (ok && w.valid()) {
            const int v_tile = w.tile;
            w.next();
            const bool has_next = w.valid();
            const int ki = 2 * t + 1;                        // load index of K(t+1)
            const int vi = has_next ? 2 * t + 2 : 2 * t + 1; // load index of V(t)
            if (has_next && !(ok = k_wait(ki % NSL))) break;
            if (has_next && need(0, w.tile)) {
                if (n_s0 > 0 && !(ok = warp_wait(BAR(B_SFREE + 0), (n_s0 - 1) & 1, abort_flag))) break;
                tc_fence_after();
                issue_s(0, ki % NSL);
                ++n_s0;
                __syncwarp();
            }
            if (!(ok = v_wait(vi % NSL))) break;
            if constexpr (KEYS != KEYS_RING)
                zero_rows<D, KT>(s_base + L::kRing + (vi % NSL) * L::kTile, zeros_from(v_tile), lane);
            if (need(0, v_tile)) {
                if (!(ok = warp_wait(BAR(B_PFULL + 0), n_p0 & 1, abort_flag))) break;
                tc_fence_after();
                issue_pv(0, vi % NSL, n_p0 == 0);
                ++n_p0;
                __syncwarp();
            }
            if (has_next) {
                if (need(1, w.tile)) {
                    if (n_s1 > 0 && !(ok = warp_wait(BAR(B_SFREE + 1), (n_s1 - 1) & 1, abort_flag))) break;
                    tc_fence_after();
                    issue_s(1, ki % NSL);
                    ++n_s1;
                }
                tc_commit_elect(BAR(B_SLOTE + ki % NSL));
                __syncwarp();
            }
            if (need(1, v_tile)) {
                if (!(ok = warp_wait(BAR(B_PFULL + 1), n_p1 & 1, abort_flag))) break;
                tc_fence_after();
                issue_pv(1, vi % NSL, n_p1 == 0);
                ++n_p1;
            }
            tc_commit_elect(BAR(B_SLOTE + vi % NSL));
            __syncwarp();
            ++t;
        }
        if (!ok && lane == 0) record_timeout(args.status, abort_flag);
        // every MMA issued above has finished before tensor memory is freed
        __syncwarp();
        tc_commit_elect(BAR(B_FINAL));
        __syncwarp();
        volatile int never = 0;
        mbar_wait(BAR(B_FINAL), 0, &never);
    } else if (warp == 1) {
        // ================================================= MMA issuers (d = 128)
        regs_shrink<LOW_REGS>();
        // Warp 1 issues the S products and warp 3 the PV products, so that a
        // wait of one never holds back the other (the tensor pipe takes only a
        // few MMAs ahead of execution).  Each commits its own products: warp 1
        // releases K slots, warp 3 V slots.
        // Per key tile t, warp 1: S_0(t+1), S_1(t+1); warp 3: PV_0(t), PV_1(t).
        // P_g goes to shared memory, so S_g(t+1) may overwrite S_g(t) in
        // tensor memory as soon as the softmax warps of tile g are done with it
        // (S free); no S product waits for a PV product.  Descriptors are built
        // once; each k-step adds a compile-time offset (16-byte units) to the
        // start-address field: 32 B per 16-element step inside a 64-column box
        // and one box (16 KB) for columns 64-127 of Q, K and P, and 16 rows
        // (2 KB) per step of V.  The whole warp runs the issue code and
        // elect.sync picks the issuing lane.
        const uint64_t dq[2] = {sdesc_sw128(s_base + L::kQ, 16, 1024),
                                sdesc_sw128(s_base + L::kQ + L::kTile, 16, 1024)};
        const uint64_t dk0 = sdesc_sw128(s_base + L::kRing, 16, KT::kGroup);
        auto issue_s = [&](int g, int slot) {
            const uint64_t a0 = dq[g], b0 = dk0 + (uint64_t)(slot * (L::kTile >> 4));
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
        auto k_wait = [&](int sl) -> bool {
            const bool got = warp_wait(BAR(B_KF + sl), (k_parity >> sl) & 1u, abort_flag);
            k_parity ^= 1u << sl;
            return got;
        };
        // the issuers need only the number of key tiles the walk visits,
        // which warp 4 counts (and, when skipping, its step table)
        bool ok = warp_wait(BAR(B_TCOUNT), 0, abort_flag);
        const int T = ok ? *tile_count : 0;
        ok = ok && warp_wait(BAR(B_QFULL), 0, abort_flag);
        if constexpr (!SKIP) {
            int t = 0;
            Walk w = walk0;
            if constexpr (EDGES) w.start_step();
            const SeenTiles seen0 = seen_by(0), seen1 = seen_by(1);
            int n0 = 0, n1 = 0;   // S products issued per Q tile
            if (ok && T > 0) {
                ok = k_wait(0);   // K(0) is load 0
                tc_fence_after();
                if (ok) {
                    if (!EDGES || seen0.has(w_tile(w))) {
                        issue_s(0, 0);
                        ++n0;
                    }
                    if (EDGES ? seen1.has(w_tile(w)) : two_tiles) {
                        issue_s(1, 0);
                        ++n1;
                    }
                    tc_commit_elect(BAR(B_SLOTE + 0));
                }
                __syncwarp();
            }
#pragma unroll 1
            for (; ok && t + 1 < T; ++t) {
                const int ki = 2 * t + 1;                    // load index of K(t+1)
                if constexpr (EDGES) w.next();
                if (!(ok = k_wait(ki % NSL))) break;
                if (!EDGES || seen0.has(w_tile(w))) {
                    if ((!EDGES || n0 > 0) &&
                        !(ok = warp_wait(BAR(B_SFREE + 0), (EDGES ? n0 - 1 : t) & 1, abort_flag))) break;
                    tc_fence_after();
                    issue_s(0, ki % NSL);
                    ++n0;
                    __syncwarp();
                }
                if (EDGES ? seen1.has(w_tile(w)) : two_tiles) {
                    if ((!EDGES || n1 > 0) &&
                        !(ok = warp_wait(BAR(B_SFREE + 1), (EDGES ? n1 - 1 : t) & 1, abort_flag))) break;
                    tc_fence_after();
                    issue_s(1, ki % NSL);
                    ++n1;
                }
                tc_commit_elect(BAR(B_SLOTE + ki % NSL));
                __syncwarp();
            }
        } else {
            // S_g is issued only for the tiles Q tile g needs; each group's
            // S-free wait counts that group's own products.  A K slot is
            // released after its tile, whether or not any S read it.
            StepCursor cs;
            cs.start((ok && *tab_ok) ? step_tab : nullptr, args.num_steps);
            int ks0 = 0, ks1 = 0;         // S products issued per Q tile
            if (ok && T > 0) {
                ok = k_wait(0);   // K(0) is load 0
                tc_fence_after();
                if (ok) {
                    if (cs.need(0)) {
                        issue_s(0, 0);
                        ++ks0;
                    }
                    if (cs.need(1)) {
                        issue_s(1, 0);
                        ++ks1;
                    }
                    tc_commit_elect(BAR(B_SLOTE + 0));
                }
                __syncwarp();
            }
#pragma unroll 1
            for (int t = 0; ok && t + 1 < T; ++t) {
                cs.next();
                const int ki = 2 * t + 1;                    // load index of K(t+1)
                if (!(ok = k_wait(ki % NSL))) break;
                if (cs.need(0)) {
                    if (ks0 > 0 && !(ok = warp_wait(BAR(B_SFREE + 0), (ks0 - 1) & 1, abort_flag))) break;
                    tc_fence_after();
                    issue_s(0, ki % NSL);
                    ++ks0;
                    __syncwarp();
                }
                if (cs.need(1)) {
                    if (ks1 > 0 && !(ok = warp_wait(BAR(B_SFREE + 1), (ks1 - 1) & 1, abort_flag))) break;
                    tc_fence_after();
                    issue_s(1, ki % NSL);
                    ++ks1;
                }
                tc_commit_elect(BAR(B_SLOTE + ki % NSL));
                __syncwarp();
            }
        }
        if (!ok && lane == 0) record_timeout(args.status, abort_flag);
        // every MMA this warp issued has finished before tensor memory is freed
        __syncwarp();
        tc_commit_elect(BAR(B_FINAL));
        __syncwarp();
        volatile int never = 0;
        mbar_wait(BAR(B_FINAL), 0, &never);
    } else if (warp == 3 && TWO_ISSUERS) {
        // ================================================= MMA issuer for PV (see warp 1)
        regs_shrink<LOW_REGS>();
        const uint64_t dp[2] = {sdesc_sw128(s_base + L::kP, 16, 1024),
                                sdesc_sw128(s_base + L::kP + 2 * L::kBox, 16, 1024)};
        const uint64_t dv0 = sdesc_sw128(s_base + L::kRing, KT::kHalf, KT::kGroup);
        auto issue_pv = [&](int g, int slot, bool first) {
            constexpr uint32_t hb = L::kBox >> 4;
            const uint64_t a0 = dp[g], b0 = dv0 + (uint64_t)(slot * (L::kTile >> 4));
            const uint32_t d = tmem + 256 + g * D;
            constexpr uint32_t vs = KT::kStep;
            mma_ss_elect<0, 0>(d, a0, b0, IDESC_O, first ? 0u : 1u);
            mma_ss_elect<2, vs>(d, a0, b0, IDESC_O, 1u);
            mma_ss_elect<4, 2 * vs>(d, a0, b0, IDESC_O, 1u);
            mma_ss_elect<6, 3 * vs>(d, a0, b0, IDESC_O, 1u);
            mma_ss_elect<hb, 4 * vs>(d, a0, b0, IDESC_O, 1u);
            mma_ss_elect<hb + 2, 5 * vs>(d, a0, b0, IDESC_O, 1u);
            mma_ss_elect<hb + 4, 6 * vs>(d, a0, b0, IDESC_O, 1u);
            mma_ss_elect<hb + 6, 7 * vs>(d, a0, b0, IDESC_O, 1u);
            tc_commit_elect(BAR(B_PVDONE + g));
        };
        uint32_t v_parity = 0;   // bit s: parity of the next V load of slot s
        auto v_wait = [&](int sl) -> bool {
            const bool got = warp_wait(BAR(B_VF + sl), (v_parity >> sl) & 1u, abort_flag);
            v_parity ^= 1u << sl;
            return got;
        };
        // the issuers need only the number of key tiles the walk visits,
        // which warp 4 counts (and, when skipping, its step table)
        bool ok = warp_wait(BAR(B_TCOUNT), 0, abort_flag);
        const int T = ok ? *tile_count : 0;
        ok = ok && warp_wait(BAR(B_QFULL), 0, abort_flag);
        if constexpr (!SKIP) {
            int t = 0;
            Walk wv = walk0;
            if constexpr (KEYS != KEYS_RING) wv.start_step();
            const SeenTiles seen0 = seen_by(0), seen1 = seen_by(1);
            int n0 = 0, n1 = 0;   // PV products issued per Q tile
#pragma unroll 1
            for (; ok && t < T; ++t) {
                const bool has_next = t + 1 < T;
                const int vi = has_next ? 2 * t + 2 : 2 * t + 1; // load index of V(t)
                if (!(ok = v_wait(vi % NSL))) break;
                if constexpr (KEYS != KEYS_RING)
                    zero_rows<D, KT>(s_base + L::kRing + (vi % NSL) * L::kTile, zeros_from(wv.tile), lane);
                if (!EDGES || seen0.has(w_tile(wv))) {
                    if (!(ok = warp_wait(BAR(B_PFULL + 0), (EDGES ? n0 : t) & 1, abort_flag))) break;
                    tc_fence_after();
                    issue_pv(0, vi % NSL, EDGES ? n0 == 0 : t == 0);
                    ++n0;
                    __syncwarp();
                }
                if (EDGES ? seen1.has(w_tile(wv)) : two_tiles) {
                    if (!(ok = warp_wait(BAR(B_PFULL + 1), (EDGES ? n1 : t) & 1, abort_flag))) break;
                    tc_fence_after();
                    issue_pv(1, vi % NSL, EDGES ? n1 == 0 : t == 0);
                    ++n1;
                }
                tc_commit_elect(BAR(B_SLOTE + vi % NSL));
                __syncwarp();
                if constexpr (KEYS != KEYS_RING) wv.next();
            }
        } else {
            // PV_g only for the tiles Q tile g needs; P-full waits and the
            // accumulate flag count that group's own products
            StepCursor cv;
            cv.start((ok && *tab_ok) ? step_tab : nullptr, args.num_steps);
            int kv0 = 0, kv1 = 0;         // PV products issued per Q tile
#pragma unroll 1
            for (int t = 0; ok && t < T; ++t) {
                const bool has_next = t + 1 < T;
                const int vi = has_next ? 2 * t + 2 : 2 * t + 1; // load index of V(t)
                if (!(ok = v_wait(vi % NSL))) break;
                if (cv.need(0)) {
                    if (!(ok = warp_wait(BAR(B_PFULL + 0), kv0 & 1, abort_flag))) break;
                    tc_fence_after();
                    issue_pv(0, vi % NSL, kv0 == 0);
                    ++kv0;
                    __syncwarp();
                }
                if (cv.need(1)) {
                    if (!(ok = warp_wait(BAR(B_PFULL + 1), kv1 & 1, abort_flag))) break;
                    tc_fence_after();
                    issue_pv(1, vi % NSL, kv1 == 0);
                    ++kv1;
                }
                tc_commit_elect(BAR(B_SLOTE + vi % NSL));
                __syncwarp();
                cv.next();
            }
        }
        if (!ok && lane == 0) record_timeout(args.status, abort_flag);
        // every MMA this warp issued has finished before tensor memory is freed
        __syncwarp();
        tc_commit_elect(BAR(B_FINAL));
        __syncwarp();
        volatile int never = 0;
        mbar_wait(BAR(B_FINAL), 0, &never);
    } else if (warp < 4) {
        regs_shrink<LOW_REGS>();
    } else {
        // ================================================= softmax
        regs_grow<216>();
        if (TWO_ISSUERS && warp == 4) {
            // the number of key tiles of the walk, one ring step per lane, for
            // the two MMA issuers (the S issuer waits for it before S(0)).  The
            // tile-skipping variant also writes the step table: for each ring
            // step (one lane per step) the unit's key-tile range and each Q
            // tile's own range inside it, from its first row's sequence start
            // to its last row (or that row's sequence end without the causal
            // mask).  Past kMaxSteps steps there is no table and every tile
            // counts for both Q tiles.
            int T = 0;
            bool have_tab = false;
            if constexpr (SKIP) have_tab = args.num_steps <= L::kMaxSteps;
            if constexpr (KEYS != KEYS_RING) {
                T = walk0.end - walk0.i;
            } else if (have_tab) {
                int64_t glo_pos[2], ghi_pos[2];
                bool gvalid[2];
#pragma unroll
                for (int gg = 0; gg < 2; ++gg) {
                    const int fr = row0 + 128 * gg, lrow = min(S, fr + 128) - 1;
                    gvalid[gg] = fr < S;
                    int64_t unused;
                    row_key_bounds(args.cu_seqlens, args.n_seqs, (int64_t)N * S,
                                   token_pos(args.layout, q_rank, gvalid[gg] ? fr : 0, N, S), args.causal,
                                   glo_pos[gg], unused);
                    row_key_bounds(args.cu_seqlens, args.n_seqs, (int64_t)N * S,
                                   token_pos(args.layout, q_rank, gvalid[gg] ? lrow : 0, N, S), args.causal,
                                   unused, ghi_pos[gg]);
                }
                for (int s0 = 0; s0 < args.num_steps; s0 += 32) {
                    const int st = s0 + lane;
                    int cnt = 0;
                    if (st < args.num_steps) {
                        const int j = walk0.kv_fixed >= 0 ? walk0.kv_fixed
                                                          : ((q_rank - st - walk0.step_base) % N + N) % N;
                        int e[6];
                        step_tile_ranges(args.layout, N, S, j, walk0.lo_pos, walk0.hi_pos, glo_pos, ghi_pos,
                                         gvalid, e);
#pragma unroll
                        for (int c = 0; c < 6; ++c) step_tab[6 * st + c] = e[c];
                        cnt = e[1] - e[0];
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) cnt += __shfl_xor_sync(0xffffffffu, cnt, o);
                    T += cnt;
                }
            } else {
                // one lane per ring step, summed over the warp
                for (int s0 = 0; s0 < args.num_steps; s0 += 32) {
                    int cnt = s0 + lane < args.num_steps ? walk0.step_tiles(s0 + lane) : 0;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) cnt += __shfl_xor_sync(0xffffffffu, cnt, o);
                    T += cnt;
                }
            }
            __syncwarp();
            if (lane == 0) {
                *tile_count = T;
                if constexpr (SKIP) *tab_ok = have_tab ? 1 : 0;
                mbar_arrive(BAR(B_TCOUNT));
            }
            __syncwarp();
        }
        const int g = (warp - 4) >> 2;
        const int wq = warp & 3;
        const int r = wq * 32 + lane;                 // row inside Q tile g (= TMEM lane)
        const int a = row0 + g * 128 + r;             // local query row in the shard
        const int a_c = a < S ? a : S - 1;
        const int64_t my_pos = token_pos(args.layout, q_rank, a_c, N, S);
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        const uint32_t tS = tmem + lane_off + g * 128;
        const uint32_t tO = tmem + lane_off + 256 + g * D;
        const float sl2 = args.scale_log2;

        float m_ref = 0.f;        // reference point of the exponentials (log2 units)
        float l = 0.f;            // running denominator, relative to m_ref
        float lr = 0.f;           // the same sum over the bf16-rounded P the MMA uses
        int64_t my_lo_pos = 0, my_hi_pos = 0;
        RowKeys rk{};
        if constexpr (KEYS == KEYS_RING)
            row_key_bounds(args.cu_seqlens, args.n_seqs, (int64_t)N * S, my_pos, args.causal, my_lo_pos, my_hi_pos);
        else if constexpr (KEYS == KEYS_WINDOW)
            rk = window_row(args.cu_seqlens, args.n_seqs, S, a_c, args.window, args.sinks);
        // KEYS_PAGED: row r is token r / group of the Q tile; rows past the
        // tile's tokens or the unit's take the last token's keys, so that no
        // tile is masked for their sake, and are not stored
        bool live = KEYS != KEYS_WINDOW || a < row_end;     // the row is stored
        bool warp_live = true;      // some row of the warp is
        int my_tok = 0;
        if constexpr (KEYS == KEYS_PAGED) {
            const int tok = r / args.seqs.group;
            my_tok = g * args.tile_tokens + tok;
            live = tok < args.tile_tokens && my_tok < pu.n;
            warp_live = __any_sync(0xffffffffu, live);
            rk = paged_row(args.seqs, pu.p0 + min(my_tok, pu.n - 1));
        }
        Walk w = walk0;
        w.start_step();
        int t = 0;              // key tiles this Q tile has processed
        bool ok = true;
        bool have_tab = false;  // tile skipping: the step table was written
        if constexpr (SKIP) {
            ok = warp_wait(BAR(B_TCOUNT), 0, abort_flag);
            have_tab = ok && *tab_ok != 0;
        }
        int cur_step = -1;
        int klo = 0, khi = S;   // this row's visible local keys [klo, khi) of shard w.j
        // (t counts the tiles processed: without skipping, every tile the walk visits)
        const SeenTiles seen_g = seen_by(g);
        // (with EDGES, and with SKIP, t counts the tiles this Q tile took)
        for (; (!(SKIP || EDGES) || ok) && w.valid(); w.next(), t += SKIP || EDGES ? 0 : 1) {
            if constexpr (EDGES) {
                if (!seen_g.has(w.tile)) continue;
            }
            if constexpr (KEYS == KEYS_PAGED) {
                if (g == 1 && !two_tiles) break;
                if (!warp_live) {
                    // no row here is stored: its P may be anything
                    if (!(ok = warp_wait(BAR(B_SFULL + g), t & 1, abort_flag))) break;
                    mbar_arrive(BAR(B_SFREE + g));
                    if (t > 0 && !(ok = warp_wait(BAR(B_PVDONE + g), (t - 1) & 1, abort_flag))) break;
                    mbar_arrive(BAR(B_PFULL + g));
                    continue;
                }
            }
            if constexpr (KEYS != KEYS_RING) {
                klo = rk.lo;
                khi = rk.hi;
            } else if (w.step != cur_step) {
                cur_step = w.step;
                klo = (int)keys_upto(args.layout, w.j, my_lo_pos, N, S);
                khi = (int)keys_upto(args.layout, w.j, my_hi_pos, N, S);
            }
            // a tile no row of this Q tile sees (the tiles of shard w.j it
            // sees are [e[0], e[1])): the MMA issuers skip its S and PV too
            if constexpr (SKIP) {
                if (have_tab) {
                    const int *e = step_tab + 6 * w.step + 2 + 2 * g;
                    if (w.tile < e[0] || w.tile >= e[1]) continue;
                }
            }
            if (!(ok = warp_wait(BAR(B_SFULL + g), t & 1, abort_flag))) break;
            tc_fence_after();
            const int lim = khi - w.tile * 128;       // columns [lim_lo, lim) are visible
            const int lim_lo = klo - w.tile * 128;
            // windowed rows also see the sink columns [sk_lo, sk_hi)
            const int sk_lo = KEYS == KEYS_RING ? 0 : rk.slo - w.tile * 128;
            const int sk_hi = KEYS == KEYS_RING ? 0 : rk.shi - w.tile * 128;
            const bool partial = lim < 128 || lim_lo > 0;
            uint32_t sr[4][32];
            auto load_s = [&]() {
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld32(tS + q * 32, sr[q]);
                tmem_wait_ld();
                if (__any_sync(0xffffffffu, partial)) {
                    // the warp's rows see columns [lim_lo, lim) each; a 32-column
                    // chunk inside [largest lim_lo, smallest lim) is visible to
                    // every row of the warp and needs no mask (a warp's limits
                    // differ by about one column per row, so at most two chunks
                    // of a tile are masked element by element)
                    const int hi_min = (int)__reduce_min_sync(0xffffffffu, (unsigned)min(max(lim, 0), 128));
                    const int lo_max = (int)__reduce_max_sync(0xffffffffu, (unsigned)min(max(lim_lo, 0), 128));
                    float *s = reinterpret_cast<float *>(&sr[0][0]);
                    if constexpr (KEYS == KEYS_RING) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if (32 * q >= lo_max && 32 * q + 32 <= hi_min) continue;
#pragma unroll
                            for (int c = 32 * q; c < 32 * q + 32; ++c)
                                if (c >= lim || c < lim_lo) s[c] = -INFINITY;
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if (32 * q >= lo_max && 32 * q + 32 <= hi_min) continue;
                            // bit c: column 32 q + c is visible
                            const uint32_t seen = (low_bits(lim - 32 * q) & ~low_bits(lim_lo - 32 * q)) |
                                                  (low_bits(sk_hi - 32 * q) & ~low_bits(sk_lo - 32 * q));
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(seen & (1u << c))) s[32 * q + c] = -INFINITY;
                        }
                    }
                }
            };
            // P is computed against the current reference point and kept in
            // registers until the row's denominator has been checked; only
            // when it would leave [kSumLo, kSumHi] (or is not a number) does the
            // warp reload S (still intact in tensor memory), move the
            // reference to max(tile max, reference + log2 l) -- the sum then
            // lies in [1, 129] -- rescale O, l and lr, and compute P again.
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
                bool bad = !(ln >= kSumLo && ln <= kSumHi);
                // a windowed row may see no column of a tile its unit visits:
                // nothing is added and nothing has to move
                if constexpr (KEYS != KEYS_RING)
                    bad = bad && live && (max(lim_lo, 0) < min(lim, 128) || max(sk_lo, 0) < min(sk_hi, 128));
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
                    // a row that has summed nothing yet has nothing to rescale (and
                    // its factor may pass 2^128, where 0 would become NaN)
                    const float alpha = l > 0.f ? ex2(m_ref - m_new) : 1.f;
                    l *= alpha;
                    lr *= alpha;
                    m_ref = m_new;
                    // O holds PV of every earlier tile once PV_g(t-1) is done;
                    // the whole warp takes part in the reload
                    if (t > 0) {
                        if (!(ok = warp_wait(BAR(B_PVDONE + g), (t - 1) & 1, abort_flag))) break;
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
                        // PV_g(t) accumulates into O only after P full, which
                        // follows the fence below
                        tmem_wait_st();
                    }
                    p_pass();
                }
            }
            l += lt;
            lr += lrt;
            // S_g(t) is no longer needed: the next S_g may overwrite it
            tc_fence_before();
            mbar_arrive(BAR(B_SFREE + g));
            // P_g(t) goes to shared memory -- the K-major A operand of PV in the
            // 128-byte-swizzled layout a TMA box load would give (16-byte chunk
            // j of row r at chunk j ^ (r mod 8); keys 0-63 in the first box) --
            // or, at d = 64, to its tensor-memory columns, once PV_g(t-1) has
            // read P_g(t-1) there
            if (t > 0 && !(ok = warp_wait(BAR(B_PVDONE + g), (t - 1) & 1, abort_flag))) break;
            if constexpr (P_IN_TMEM) {
                // the row's 128 keys as 64 packed columns (key c in the low half
                // of column c / 2), the layout a TS product reads A in
                const uint32_t tP = tmem + lane_off + 384 + g * 64;
                tmem_st32(tP, *reinterpret_cast<const uint32_t(*)[32]>(&pr[0][0]));
                tmem_st32(tP + 32, *reinterpret_cast<const uint32_t(*)[32]>(&pr[2][0]));
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(BAR(B_PFULL + g));
                if constexpr (SKIP || EDGES) ++t;
                continue;
            }
            {
                // row base (1024-byte aligned group + 128 bytes per row) and the
                // row's chunk swizzle; both are recomputed every tile rather than
                // kept live across the loop
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
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(BAR(B_PFULL + g));
            if constexpr (SKIP || EDGES) ++t;
        }
        const int T = t;
        if (!ok) {
            if (lane == 0) record_timeout(args.status, abort_flag);
        } else if (T > 0) {
            ok = warp_wait(BAR(B_PVDONE + g), (T - 1) & 1, abort_flag);
            if (!ok && lane == 0) record_timeout(args.status, abort_flag);
            tc_fence_after();
        }
        // O_g / l goes out through shared memory and TMA: staged in this
        // group's P buffer (and, for fp32 O at d = 128, its Q tile), both free
        // once PV_g(T-1) is done, as boxes of 128 rows x 128 bytes in the
        // 128-byte swizzle (16-byte chunk j of row r at chunk j ^ (r mod 8)).
        // A unit that sees no key writes O = 0.  Every warp of the group
        // reaches the barrier; after a timeout nothing is stored.
        constexpr int CPB = OUT_F32 ? 32 : 64;       // O columns per box
        constexpr int NBOX = D / CPB;
        auto box_addr = [&](int bx) -> uint32_t {
            return bx < 2 ? s_base + L::kP + g * 2 * L::kBox + bx * L::kBox
                          : s_base + L::kQ + g * L::kTile + (bx - 2) * L::kBox;
        };
        const float inv_l = lr > 0.f ? 1.f / lr : 0.f;
        if (ok) {
            const uint32_t xr = (uint32_t)(r & 7) << 4;
            const uint32_t row_off = (r >> 3) * 1024 + (r & 7) * 128;
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                if (T > 0) {
                    tmem_ld32(tO + q * 32, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int c = 0; c < 32; ++c) o[c] = 0u;
                }
                if (OUT_F32) {
                    // 32 columns = one box, eight 16-byte chunks
                    const uint32_t row = box_addr(q) + row_off;
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(row + (((uint32_t)c << 4) ^ xr)),
                                     "f"(__uint_as_float(o[4 * c]) * inv_l), "f"(__uint_as_float(o[4 * c + 1]) * inv_l),
                                     "f"(__uint_as_float(o[4 * c + 2]) * inv_l), "f"(__uint_as_float(o[4 * c + 3]) * inv_l)
                                     : "memory");
                } else {
                    // 32 columns = half a box, four 16-byte chunks
                    const uint32_t row = box_addr(q >> 1) + row_off;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t w0 = pack_bf16x2(__uint_as_float(o[8 * c + 0]) * inv_l, __uint_as_float(o[8 * c + 1]) * inv_l);
                        const uint32_t w1 = pack_bf16x2(__uint_as_float(o[8 * c + 2]) * inv_l, __uint_as_float(o[8 * c + 3]) * inv_l);
                        const uint32_t w2 = pack_bf16x2(__uint_as_float(o[8 * c + 4]) * inv_l, __uint_as_float(o[8 * c + 5]) * inv_l);
                        const uint32_t w3 = pack_bf16x2(__uint_as_float(o[8 * c + 6]) * inv_l, __uint_as_float(o[8 * c + 7]) * inv_l);
                        const uint32_t chunk = (uint32_t)((q & 1) * 4 + c);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((chunk << 4) ^ xr)),
                                     "r"(w0), "r"(w1), "r"(w2), "r"(w3)
                                     : "memory");
                    }
                }
            }
        }
        // KEYS_WINDOW: a Q tile that ends behind the last sequence goes out row by row
        const bool ragged = KEYS == KEYS_WINDOW && S < args.S && row0 + 128 * g + 128 > S;
        if (KEYS == KEYS_PAGED || ragged) {
            // each warp copies its own rows out: final rows of [T, H, d], or
            // this part's rows (fp32) for the join
            const float lse = l > 0.f ? (m_ref + lg2(l)) * 0.6931471805599453f : -INFINITY;
            const int head = h * args.seqs.group + r % args.seqs.group;
            long long at = -1;       // the row's first element
            if (KEYS == KEYS_WINDOW) {
                if (ok && live) at = (long long)((((size_t)b * args.S + a) * H + h) * D);
            } else if (ok && live && (g == 0 || two_tiles)) {
                const size_t part_row = (((size_t)unit_no * args.seqs.Hkv + h) * args.seqs.num_splits + part) *
                                            paged_unit_rows(args.seqs) +
                                        my_tok * args.seqs.group + r % args.seqs.group;
                const size_t tok = (size_t)(pu.t0 + my_tok);
                at = (long long)((split ? part_row : tok * args.seqs.H + head) * D);
                if (split) args.part_lse[part_row] = lse;
                else if (args.lse) args.lse[(size_t)head * args.seqs.T + tok] = lse;
            }
            __syncwarp();
            auto staged = [&](int row, int ch) -> uint4 {     // 16-byte chunk ch of the warp's row
                const int rr = wq * 32 + row;
                const uint32_t src = box_addr(ch >> 3) + (rr >> 3) * 1024 + (rr & 7) * 128 + (((ch & 7) ^ (rr & 7)) << 4);
                uint4 x;
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(src) : "memory");
                return x;
            };
            // rows of the staged type, or (a unit of one part in a split call) rounded to bf16 here
            const bool round = OUT_F32 && args.o_bf16 && !split;
            uint8_t *out = split ? reinterpret_cast<uint8_t *>(args.part_o) : static_cast<uint8_t *>(args.o);
            const int esz = OUT_F32 && !round ? 4 : 2;
            const int cpr = D * esz / 16;            // 16-byte chunks per row
            if ((KEYS == KEYS_WINDOW || warp_live) && *abort_flag == 0) {
#pragma unroll 4
                for (int e = lane; e < 32 * cpr; e += 32) {
                    const int row = e / cpr, ch = e % cpr;
                    const long long dst = __shfl_sync(0xffffffffu, at, row);
                    uint4 x;
                    if (round) {
                        const uint4 lo = staged(row, 2 * ch), hi = staged(row, 2 * ch + 1);
                        x.x = pack_bf16x2(__uint_as_float(lo.x), __uint_as_float(lo.y));
                        x.y = pack_bf16x2(__uint_as_float(lo.z), __uint_as_float(lo.w));
                        x.z = pack_bf16x2(__uint_as_float(hi.x), __uint_as_float(hi.y));
                        x.w = pack_bf16x2(__uint_as_float(hi.z), __uint_as_float(hi.w));
                    } else {
                        x = staged(row, ch);
                    }
                    if (dst >= 0) *reinterpret_cast<uint4 *>(out + (size_t)dst * esz + ch * 16) = x;
                }
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        if constexpr (KEYS != KEYS_PAGED) named_barrier_sync(1 + g, 128);
        if (KEYS != KEYS_PAGED && !ragged && !(KEYS == KEYS_WINDOW && row0 + 128 * g >= row_end) && wq == 0 &&
            lane == 0 && *abort_flag == 0) {
            // rows past the shard's end fall outside the tensor and are not written
            int c1, c2, c3;
            tile_coords(args.seq_order, args.layout, args.S, args.N, ring ? qi : 0, b, row0 + 128 * g, c1, c2, c3);
#pragma unroll
            for (int bx = 0; bx < NBOX; ++bx) tma_store_4d(&tmo, box_addr(bx), h * D + bx * CPB, c1, c2, c3);
            tma_store_commit();
            tma_store_wait_read();
        }
        if (KEYS != KEYS_PAGED && ok && (KEYS == KEYS_WINDOW ? live : a < S)) {
            // shard stacks: [N or 1, B, H, S]; sequence order: [B, H, L] at the row's position
            const size_t at = args.seq_order ? ((size_t)b * H + h) * ((size_t)N * S) + (size_t)my_pos
                                             : ((size_t)zq * H + h) * args.S + a;
            args.lse[at] = l > 0.f ? (m_ref + lg2(l)) * 0.6931471805599453f : -INFINITY;
        }
    }

    // ---- teardown: every role is here, all tensor-core work has finished
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace ra
