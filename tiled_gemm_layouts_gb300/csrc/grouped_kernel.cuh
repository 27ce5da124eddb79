// grouped_kernel.cuh -- products in which every group of rows has a matrix of
// its own, on sm_103a: the experts' products and their gradients.
//
//   GROUPED_ROWS     Y[i] = epilogue(X[source(i)] B[g])        rows i of group g
//   GROUPED_WEIGHT   dB[g] = sum over them of X[source(i)]^T dY[i]
//
// The main loop is that of the GEMM kernel: TMA producers fill a ring of
// 128B-swizzled stages, one thread issues tcgen05.mma into a double-buffered
// fp32 accumulator in TMEM, eight epilogue warps drain it while the next
// tile's products run; tiles of 256 x BN on a CTA pair, or 128 x BN on one CTA.
//
// Groups.  Only the device knows how many rows a group has.  Workers walk the
// same list of tiles, group by group, each taking every `workers`-th: a warp
// reads 128 groups' offsets at a time, one scan over its lanes gives their
// first tiles, a ballot the group of a tile.  Nothing is planned by another
// kernel or kept between calls.
//
// Rows by a list are fetched where they stand; no gathered copy of X is
// written (at 65536 rows of 4096 columns that would be 1.07 GB more traffic).
// With LIST three warps of their own fetch them, 16 bytes per thread and
// asynchronous copy, into the swizzled layout that a box would have, and a fourth
// hands them over to the MMA (65536 rows, 64 groups, 4096 x 1024: 373 us,
// consecutive rows 337).  Gathering TMA copies of four rows, which would need none
// of these, take about 80 cycles of the copy engine for 512 bytes, and a stage of 128
// rows 2600 where its products take 512: 1184 us.  Without LIST a part of a tile
// without rows is not fetched at all: what is left in its stage only reaches
// accumulator rows that are not stored.
//
// In GROUPED_WEIGHT the rows are the contraction, and a group's last K-block is
// ragged: it is fetched by row number from both operands (by gathering copies where
// there is no list), with zeros for the rows that are none of the group's (a box
// would bring the next group's rows, whose infinities a zero in the other operand
// does not undo).  The gathering copies make a ragged end dear: 64 groups of 1024 rows,
// 4096 x 1024, take 335 us, of 1025 rows 396 and of 1000 rows 420.
//
// Every wait is bounded; on a timeout the status word is set, copies and MMAs
// in flight are drained, TMEM is freed and the kernel returns.
#pragma once

#include "ce_kernel.cuh"
#include "direct.cuh"
#include "gemm_kernel.cuh"
#include "grouped_params.h"

namespace tg {

constexpr int kGrEpiWarps = 8;   // two per TMEM lane quadrant, each with half of a tile's columns
constexpr int kGrWarps = 3 + kGrEpiWarps;  // producers (warps 0 and 10), MMA (1), epilogue (2..9)
constexpr int kListWarps = 3;              // with LIST, behind them, and a warp that hands over what they fetched
// K-blocks per barrier transaction, one after the other in the ring.  Where an
// operand's columns are contiguous, they interleave: 64 columns of all their
// rows, then the next 64.  Two take half the copies and waits of one: the
// gradient of 65536 rows, 64 groups, 4096 x 1024, 414 us with one, 335 with two.
// Rows by a list for tiles of a pair come faster one by one: 361 us, 385.
template <int MODE, bool PAIR, bool LIST>
constexpr int kGrBlocks = MODE == GROUPED_ROWS && PAIR && LIST ? 1 : 2;
constexpr int kGrOrder = 512;              // groups that GROUPED_WEIGHT sorts by their rows
// What a K-block adds to the epilogue's time limit.  Its wait covers a tile's whole
// contraction, of up to 2^24 K-blocks, which at 250 to 900 cycles each may take longer than
// one limit; all other waits are for single K-blocks or a tile's output.
constexpr long long kGrBlockCycles = 8192;
template <bool LIST>
constexpr int kGrThreads = 32 * (kGrWarps + (LIST ? kListWarps + 1 : 0));

template <int MODE, int BN, bool PAIR, bool LIST>
struct GroupedShape : TileShape<BN, PAIR> {
    using TS = TileShape<BN, PAIR>;
    static constexpr int kUnit = 4096;  // staging per epilogue warp: 32 rows of 128 bytes
    static constexpr int kFit = (TS::kSmemLimit - 1024 - 256 - kGrEpiWarps * kUnit) / TS::kStage;
    static constexpr int kSlots = (kFit > 8 ? 8 : kFit) & ~1;
    static constexpr int kBlocks = kGrBlocks<MODE, PAIR, LIST>;
    static constexpr int kGroups = kSlots / kBlocks;  // of slots, a transaction each
    static constexpr int kGrSmemBytes =
        1024 + kSlots * TS::kStage + kGrEpiWarps * kUnit + kGrOrder * 2 + (2 * kGroups + kSlots + 5) * 8 + 16;
    static_assert(kSlots >= kListWarps && kGrSmemBytes <= TS::kSmemLimit, "shared memory budget");
};

// Gathers rows r[0..3], columns c .. c+63, as four consecutive 128-byte rows.
template <bool PAIR>
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c,
                                            const int (&r)[4]) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
            ".cta_group::2 [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
            : "memory");
}

// Source of a list's row r; a number outside the matrix for one that has none.
__device__ __forceinline__ int source_of(const GroupedRows& s, int r) {
    return r < 0 ? s.count : (int)((uint64_t)(uint32_t)r * s.magic >> s.shift);
}
// 16 bytes, of which `bytes` are read and the rest zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Arrives on the barrier once this thread's copies so far have landed.
__device__ __forceinline__ void copy16_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copy16_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Arrives on the leader CTA's barrier; what this thread knows to be written to
// its CTA's shared memory comes before.  (A release of all memory at cluster
// scope waits 1200 cycles here, of shared memory alone next to nothing.)
__device__ __forceinline__ void arrive_on_leader_release(uint32_t bar) {
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
    arrive_on_leader(bar);
}

struct GroupedItem {
    int g, lo, cnt;  // group, its first row, its rows
    int tm, tn;
};

// The tiles of one worker, in order.  Called by whole warps; every lane gets
// the same item.
template <int MODE>
struct GroupedItems {
    const GroupedParams& p;
    const uint16_t* order;   // GROUPED_WEIGHT: groups, the one with the most rows first, or null
    int lane, bm, t, step;   // GROUPED_WEIGHT: t counts rounds
    int worker;
    int window, base, incl;  // groups from `window`, their first tile, tiles up to this lane's last group
    int lo[4], cnt[4];       // this lane's four groups
    bool started;

    __device__ __forceinline__ GroupedItems(const GroupedParams& params, const uint16_t* sorted, int self, int workers,
                                            int rows_per_tile)
        : p(params), order(sorted), lane(threadIdx.x & 31), bm(rows_per_tile), t(MODE == GROUPED_WEIGHT ? 0 : self),
          step(workers), worker(self), window(-128), base(0), incl(0), started(false) {}

    __device__ __forceinline__ int bound(int g) const {
        return max(0, min(p.offset[g], p.rows));
    }
    __device__ __forceinline__ int tiles_of(int k) const { return (cnt[k] + bm - 1) / bm * p.tiles_n; }
    __device__ __forceinline__ void place(GroupedItem& it, int i, int tiles_m) const {
        const int group = p.group_m * p.tiles_n;
        const int first = i / group * p.group_m;
        const int gm = min(tiles_m - first, p.group_m), r = i - i / group * group;
        it.tm = first + r % gm;
        it.tn = r / gm;
    }
    __device__ __forceinline__ bool next(GroupedItem& it) {
        if constexpr (MODE == GROUPED_WEIGHT) {
            // Tiles take as long as their groups have rows.  Groups come sorted, and rounds
            // of one tile per worker alternate in direction, so that all have the same to
            // do within about one tile (64 groups of 512 to 1536 rows, multiples of 128, 4096
            // x 1024: 338 us, even groups 335; with ragged ends 425, as they come 500).
            const int per = p.tiles_m * p.tiles_n;
            const int i = t * step + (t & 1 ? step - 1 - worker : worker), at = i / per;
            if (at >= p.groups) return false;
            it.g = order ? order[at] : at;
            it.lo = bound(it.g);
            it.cnt = max(0, bound(it.g + 1) - it.lo);
            place(it, i - at * per, p.tiles_m);
            ++t;
            return true;
        } else {
            while (!started || t >= base + __shfl_sync(0xffffffffu, incl, 31)) {
                if (started) base += __shfl_sync(0xffffffffu, incl, 31);
                started = true;
                window += 128;
                if (window >= p.groups) {
                    t = 0x40000000;  // past every tile, for any further call
                    incl = 0;
                    window = 0x40000000;
                    return false;
                }
                int end[5];
#pragma unroll
                for (int k = 0; k < 5; ++k) end[k] = bound(min(window + 4 * lane + k, p.groups));
                incl = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    lo[k] = end[k];
                    cnt[k] = max(0, end[k + 1] - end[k]);
                    incl += tiles_of(k);
                }
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const int o = __shfl_up_sync(0xffffffffu, incl, d);
                    if (lane >= d) incl += o;
                }
            }
            const unsigned later = __ballot_sync(0xffffffffu, t < base + incl);
            if (!later) return false;  // (more tiles than 32 bits count: offsets that do not ascend)
            const int owner = __ffs(later) - 1;
            // its tiles before this one, group by group
            int i = t - base - (incl - (tiles_of(0) + tiles_of(1) + tiles_of(2) + tiles_of(3)));
            int k = 0, first = lo[0], rows = cnt[0];
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (k == j && i >= tiles_of(j)) {
                    i -= tiles_of(j);
                    k = j + 1;
                    first = lo[j + 1];
                    rows = cnt[j + 1];
                }
            it.g = window + 4 * owner + __shfl_sync(0xffffffffu, k, owner);
            it.lo = __shfl_sync(0xffffffffu, first, owner);
            it.cnt = __shfl_sync(0xffffffffu, rows, owner);
            place(it, __shfl_sync(0xffffffffu, i, owner), (it.cnt + bm - 1) / bm);
            t += step;
            return true;
        }
    }
};

template <int MODE, int BN, bool PAIR, bool LIST>
__global__ void __launch_bounds__(kGrThreads<LIST>, 1) grouped_kernel(const __grid_constant__ GroupedParams p) {
    using TS = GroupedShape<MODE, BN, PAIR, LIST>;
    constexpr int BLOCKS = TS::kBlocks;
    constexpr uint32_t kAtom = 8192u * BLOCKS;  // 64 contiguous columns of a transaction's rows
    constexpr bool WEIGHT = MODE == GROUPED_WEIGHT;
    constexpr int SLOTS = TS::kSlots, GROUPS = TS::kGroups;
    constexpr int CG = PAIR ? 2 : 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + SLOTS * TS::kAStage;
    uint8_t* staging = sB + SLOTS * TS::kBStage;
    uint16_t* sorted = reinterpret_cast<uint16_t*>(staging + kGrEpiWarps * TS::kUnit);
    uint64_t* full = reinterpret_cast<uint64_t*>(sorted + kGrOrder);
    uint64_t* empty = full + GROUPS;
    uint64_t* tfull = empty + GROUPS;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint64_t* landed = drain + 1;  // a slot's copies by the list's warps
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(landed + SLOTS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0;
    const bool leader = rank == 0;
    const int worker = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
    const int workers = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;
    const Watch w{abort_flag,
                  PAIR ? mapa_shared(smem_addr((const void*)abort_flag), rank ^ 1u) : 0u, PAIR,
                  p.status, p.timeout_cycles};

    if (threadIdx.x == 0) {
        if (!LIST || !p.p.row) prefetch_tensormap(&p.p.box);
        if (WEIGHT && (!LIST || !p.q.row)) prefetch_tensormap(&p.q.box);
        if (!WEIGHT) prefetch_tensormap(p.q_pairs ? &p.map_q2 : &p.map_q);
        for (int s = 0; s < GROUPS; ++s) {
            mbar_init(smem_addr(&full[s]), 1 + (LIST ? CG * BLOCKS : 0));
            mbar_init(smem_addr(&empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(&tfull[b]), 1);
            mbar_init(smem_addr(&tempty[b]), CG * kGrEpiWarps);
        }
        mbar_init(smem_addr(drain), 1);
        for (int s = 0; s < SLOTS; ++s) mbar_init(smem_addr(&landed[s]), 32);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc<CG>(smem_addr(tmem_slot), TS::kTmemCols);
        tmem_relinquish<CG>();
    }
    const bool sort = WEIGHT && p.groups > 1 && p.groups <= kGrOrder;
    if (sort) {  // (the staging buffers are free)
        int* count = reinterpret_cast<int*>(staging);
        for (int g = threadIdx.x; g < p.groups; g += kGrThreads<LIST>)
            count[g] = min(max(p.offset[g + 1], 0), p.rows) - min(max(p.offset[g], 0), p.rows);
        __syncthreads();
        for (int g = threadIdx.x; g < p.groups; g += kGrThreads<LIST>) {
            int ahead = 0;
            for (int o = 0; o < p.groups; ++o) ahead += count[o] > count[g] || (count[o] == count[g] && o < g);
            sorted[ahead] = (uint16_t)g;
        }
    }
    const uint16_t* order = sort ? sorted : nullptr;
    tc_fence_before();
    if constexpr (PAIR)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    // K-blocks of an item (a group without rows still has one, of zeros)
    auto blocks_of = [&](const GroupedItem& it) { return WEIGHT ? max(1, (it.cnt + kBK - 1) / kBK) : p.num_kb; };
    // rows of the tile that lie in CTA r
    auto rows_in = [&](const GroupedItem& it, int r) { return min(128, max(0, it.cnt - it.tm * TS::kBM - 128 * r)); };

    if (warp == 0 || warp == 2 + kGrEpiWarps) {
        // -------------------------------------------------- TMA producers
        // Warp 0 arms each transaction and fetches P, the other one fetches Q into it.
        const bool first = warp == 0;
        int grp = 0;
        uint32_t phase = 0, armed = 0, armed_parity = 0;
        GroupedItems<MODE> items(p, order, worker, workers, TS::kBM);
        GroupedItem it;
        bool ok = true;
        const GroupedRows& s = first ? p.p : p.q;
        const bool others = LIST && (WEIGHT ? s.row != nullptr : first);  // the list's warps fetch this operand
        const uint32_t dst0 = smem_addr(first ? sA : sB), block_bytes = first ? (uint32_t)TS::kAStage : (uint32_t)TS::kBStage;
        const int quad = lane & 15;  // GROUPED_WEIGHT: the rows that this lane gathers
        while (ok && items.next(it)) {
            const int num_kb = blocks_of(it);
            // bytes that the two producers of every CTA bring per K-block
            uint32_t bytes;
            if constexpr (WEIGHT) {
                bytes = (uint32_t)((LIST && p.p.row ? 0 : TS::kAStage) + (LIST && p.q.row ? 0 : TS::kBStage)) * CG;
            } else {
                auto rows_bytes = [&](int r) { return !LIST && rows_in(it, r) ? (uint32_t)TS::kAStage : 0u; };
                bytes = rows_bytes(0) + (PAIR ? rows_bytes(1) : 0u) + (p.q_mn ? 0u : (uint32_t)TS::kBStage * CG);
            }
            const int mine = rows_in(it, (int)rank);
            const int row0 = it.tm * TS::kBM + 128 * (int)rank;               // not WEIGHT
            const int c0 = first ? row0 : it.tn * BN + (int)rank * TS::kBNC;  // WEIGHT: first column of P or Q
            for (int kb = 0; kb < num_kb; kb += BLOCKS) {
                const int n = min(BLOCKS, num_kb - kb);
                const bool got = wait_bar(smem_addr(&empty[grp]), phase ^ 1, w, DEV_TIMEOUT_PRODUCER + 1);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                const uint32_t fb_local = smem_addr(&full[grp]);
                if (first && leader && lane == 0) {
                    // (a box of contiguous columns always holds both blocks' rows)
                    const uint32_t whole = !WEIGHT && p.q_mn ? (uint32_t)(BLOCKS * TS::kBStage) * CG : 0u;
                    mbar_arrive_expect_tx(fb_local, bytes * (uint32_t)n + whole);
                    armed |= 1u << grp;
                    armed_parity = (armed_parity & ~(1u << grp)) | (phase << grp);
                }
                const uint32_t fb = PAIR ? mapa_shared(fb_local, 0) : fb_local;
                const uint32_t dst = dst0 + (uint32_t)grp * BLOCKS * block_bytes;
                auto load2 = [&](uint32_t at, const CUtensorMap* map, int x, int y) {
                    if constexpr (PAIR)
                        tma_load_2d_pair(at, map, fb, x, y);
                    else
                        tma_load_2d(at, map, fb, x, y);
                };
                auto load3 = [&](uint32_t at, const CUtensorMap* map, int x, int y, int z) {
                    if constexpr (PAIR)
                        tma_load_3d_pair(at, map, fb, x, y, z);
                    else
                        tma_load_3d(at, map, fb, x, y, z);
                };
                auto load4 = [&](uint32_t at, const CUtensorMap* map, int y, int z, int u) {
                    if constexpr (PAIR)
                        tma_load_4d_pair(at, map, fb, 0, y, z, u);
                    else
                        tma_load_4d(at, map, fb, 0, y, z, u);
                };
                if (others) {
                } else if constexpr (WEIGHT) {
                    // rows of the group, in atoms of 64 columns
                    const int atoms = first ? 2 : TS::kBBoxes;
                    if ((kb + BLOCKS) * kBK <= it.cnt) {
                        if (lane < atoms) load2(dst + lane * kAtom, &s.box, c0 + 64 * lane, it.lo + kb * kBK);
                    } else {
                        for (int j = 0; j < n; ++j) {
                            int src[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int i = (kb + j) * kBK + 4 * quad + k;
                                src[k] = i < it.cnt ? it.lo + i : s.count;
                            }
                            for (int h = lane >> 4; h < atoms; h += 2)
                                tma_gather4<PAIR>(dst + h * kAtom + j * 8192 + quad * 512, &s.gather, fb, c0 + 64 * h, src);
                        }
                    }
                } else if (first) {
                    if (lane == 0 && mine > 0) {
                        if (n == 2 && kb + 2 <= s.pairs)
                            load3(dst, &s.box2, 0, it.lo + row0, kb);
                        else
                            for (int j = 0; j < n; ++j) load2(dst + j * TS::kAStage, &s.box, (kb + j) * kBK, it.lo + row0);
                    }
                } else if (p.q_mn) {
                    if (lane < TS::kBBoxes) load3(dst + lane * kAtom, &p.map_q, c0 + 64 * lane, kb * kBK, it.g);
                } else if (lane == 0) {
                    if (n == 2 && kb + 2 <= p.q_pairs)
                        load4(dst, &p.map_q2, c0, kb, it.g);
                    else
                        for (int j = 0; j < n; ++j) load3(dst + j * TS::kBStage, &p.map_q, (kb + j) * kBK, c0, it.g);
                }
                if (++grp == GROUPS) {
                    grp = 0;
                    phase ^= 1;
                }
            }
        }
        if (*abort_flag && first && lane == 0) {  // no TMA write may land after the CTA exits
            for (int q = 0; q < GROUPS; ++q)
                if (armed & (1u << q)) drain_bar(smem_addr(&full[q]), (armed_parity >> q) & 1, w);
        }
    } else if (LIST && warp >= kGrWarps && warp < kGrWarps + kListWarps) {
        // ------------------------------------------- rows by their numbers
        // Each warp takes every kListWarps-th slot: 1024 units of 16 bytes, lane's
        // unit u of every kApart-th row.  16-byte unit k of 128-byte row r lies at
        // unit k ^ (r mod 8).  The copies report to the slot's own barrier, so a warp
        // only ever waits for free slots.
        constexpr int kUnitsOfRow = WEIGHT ? 16 : 8, kApart = 32 / kUnitsOfRow, kRows = WEIGHT ? 64 : 128;
        static_assert(!WEIGHT || TS::kBNC == 128, "P's and Q's stages have one shape");
        const int self = warp - kGrWarps;
        const bool is_p = !WEIGHT || p.p.row;
        const GroupedRows& s = is_p ? p.p : p.q;
        const int u = lane % kUnitsOfRow, q = lane / kUnitsOfRow;
        const uint32_t dst0 = smem_addr(is_p ? sA : sB);
        const uint32_t stage_bytes = is_p ? (uint32_t)TS::kAStage : (uint32_t)TS::kBStage;
        // row kApart j + q: its number within eight repeats every 8 / kApart rows
        uint32_t to[8 / kApart];
#pragma unroll
        for (int j = 0; j < 8 / kApart; ++j) {
            const int r = kApart * j + q;
            to[j] = (uint32_t)((u >> 3) * kAtom + r * 128 + (((u & 7) ^ (r & 7)) << 4));
        }
        const uint16_t* base = static_cast<const uint16_t*>(s.base);
        int slot = self, wait = self;  // of this warp's next K-block; K-blocks until it is due
        uint32_t phase = 0;
        GroupedItems<MODE> items(p, order, worker, workers, TS::kBM);
        GroupedItem it;
        bool ok = true;
        while (ok && items.next(it)) {
            const int num_kb = blocks_of(it), all_kb = (num_kb + BLOCKS - 1) / BLOCKS * BLOCKS;
            const int row0 = it.tm * TS::kBM + 128 * (int)rank;                 // not WEIGHT
            const int c0 = is_p ? row0 : it.tn * BN + (int)rank * TS::kBNC;     // WEIGHT
            // lane's rows of the stage: lane, lane + 32, ...
            int src[kRows / 32], ahead[kRows / 32];
            auto fetch_rows = [&](int i0, int (&r)[kRows / 32]) {
#pragma unroll
                for (int j = 0; j < kRows / 32; ++j) r[j] = i0 + 32 * j + lane < it.cnt ? s.row[it.lo + i0 + 32 * j + lane] : -1;
            };
            auto sources = [&](const int (&r)[kRows / 32]) {
#pragma unroll
                for (int j = 0; j < kRows / 32; ++j) src[j] = source_of(s, r[j]);
            };
            // (GROUPED_WEIGHT: the next block's numbers are loaded while this one's rows are)
            fetch_rows(WEIGHT ? wait * kBK : row0, ahead);
            if (!WEIGHT) sources(ahead);
            int kb = wait;
            for (; kb < all_kb; kb += kListWarps) {
                if constexpr (WEIGHT) {
                    sources(ahead);
                    fetch_rows((kb + kListWarps) * kBK, ahead);
                }
                const bool got = wait_bar(smem_addr(&empty[slot / BLOCKS]), phase ^ 1, w, DEV_TIMEOUT_PRODUCER + 3);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                const uint32_t dst = dst0 + (uint32_t)(slot / BLOCKS) * BLOCKS * stage_bytes +
                                     (uint32_t)(slot % BLOCKS) * (WEIGHT ? 8192u : (uint32_t)TS::kAStage);
                const int col = (WEIGHT ? c0 : kb * kBK) + 8 * u;
                const uint32_t bytes = 2u * (uint32_t)min(8, max(0, s.cols - col));
                const uint16_t* from = base + (bytes ? col : 0);
                if (kb < num_kb) {
                    // (eight rows' numbers at a time: copies do not move past shuffles)
#pragma unroll
                    for (int j0 = 0; j0 < kRows / kApart; j0 += 8) {
                        const uint16_t* at[8];
                        uint32_t n[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int r = __shfl_sync(0xffffffffu, src[kApart * (j0 + j) / 32], (kApart * (j0 + j) & 31) + q);
                            n[j] = r < s.count ? bytes : 0u;
                            at[j] = from + (r < s.count ? r : 0) * s.ld;
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            copy16(dst + to[(j0 + j) % (8 / kApart)] + (j0 + j) / (8 / kApart) * 1024, at[j], n[j]);
                    }
                }
                copy16_arrive(smem_addr(&landed[slot]));
                slot += kListWarps;
                if (slot >= SLOTS) {
                    slot -= SLOTS;
                    phase ^= 1;
                }
            }
            wait = kb - all_kb;
        }
        copy16_wait_all();
    } else if (LIST && warp == kGrWarps + kListWarps) {
        // ------------------------------- from the list's warps to the MMA
        // Ordinary writes become visible to the proxy that the MMA reads through by a
        // fence after they are known to have landed.  It is a thread of its own that
        // passes it: the fence waits for every copy its thread has in flight, so a
        // warp that copied and fenced had nothing in flight meanwhile (the gradient of
        // the sizes above: 449 us with five such warps, 410 with three and this one).
        int slot = 0;
        uint32_t phase = 0;
        GroupedItems<MODE> items(p, order, worker, workers, TS::kBM);
        GroupedItem it;
        bool ok = true;
        while (ok && items.next(it)) {
            const int all_kb = (blocks_of(it) + BLOCKS - 1) / BLOCKS * BLOCKS;
            if (lane == 0) {
                for (int kb = 0; kb < all_kb; ++kb) {
                    ok = wait_bar(smem_addr(&landed[slot]), phase, w, DEV_TIMEOUT_PRODUCER + 4);
                    if (!ok) break;
                    fence_proxy_async_shared();
                    if constexpr (PAIR)
                        arrive_on_leader_release(smem_addr(&full[slot / BLOCKS]));
                    else
                        mbar_arrive(smem_addr(&full[slot / BLOCKS]));
                    if (++slot == SLOTS) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        }
    } else if (warp == 1 && leader) {
        // ---------------------------------------------------- MMA issuer
        int grp = 0;
        uint32_t phase = 0;
        bool ok = true;
        const uint32_t d_hi = smem_desc_hi_sw128(1024);
        const bool q_mn = WEIGHT || p.q_mn;
        const uint32_t a_lo0 = smem_desc_lo(smem_addr(sA), WEIGHT ? kAtom : 16u);
        const uint32_t b_lo0 = smem_desc_lo(smem_addr(sB), q_mn ? kAtom : 16u);
        constexpr uint32_t a_kstep = WEIGHT ? (2048u >> 4) : (32u >> 4);
        constexpr uint32_t a_block = (WEIGHT ? 8192u : (uint32_t)TS::kAStage) >> 4;
        const uint32_t b_kstep = q_mn ? (2048u >> 4) : (32u >> 4);
        const uint32_t b_block = (q_mn ? 8192u : (uint32_t)TS::kBStage) >> 4;
        GroupedItems<MODE> items(p, order, worker, workers, TS::kBM);
        GroupedItem it;
        for (int i = 0; ok && items.next(it); ++i) {
            const int num_kb = blocks_of(it);
            if (lane == 0) {
                const int buf = i & 1;
                ok = wait_bar(smem_addr(&tempty[buf]), ((i >> 1) & 1) ^ 1, w, DEV_TIMEOUT_MMA + 3);
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + buf * BN;
                for (int kb = 0; ok && kb < num_kb; kb += BLOCKS) {
                    ok = wait_bar(smem_addr(&full[grp]), phase, w, DEV_TIMEOUT_MMA + 4);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int j = 0; j < BLOCKS; ++j) {
                        if (kb + j >= num_kb) break;
                        const uint32_t a_lo = a_lo0 + (uint32_t)grp * (BLOCKS * TS::kAStage >> 4) + j * a_block;
                        const uint32_t b_lo = b_lo0 + (uint32_t)grp * (BLOCKS * TS::kBStage >> 4) + j * b_block;
#pragma unroll
                        for (int kk = 0; kk < kBK / kUmmaK; ++kk)
                            mma_f16<CG>(d_tmem, smem_desc_join(a_lo + kk * a_kstep, d_hi),
                                        smem_desc_join(b_lo + kk * b_kstep, d_hi), p.idesc, kb + j != 0 || kk != 0);
                    }
                    if constexpr (PAIR)
                        mma_commit_pair(smem_addr(&empty[grp]), 0x3);
                    else
                        mma_commit(smem_addr(&empty[grp]));
                    if (++grp == GROUPS) {
                        grp = 0;
                        phase ^= 1;
                    }
                }
                if (ok) {
                    if constexpr (PAIR)
                        mma_commit_pair(smem_addr(&tfull[buf]), 0x3);
                    else
                        mma_commit(smem_addr(&tfull[buf]));
                }
            }
            ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        }
        if (lane == 0) {  // nothing may still write TMEM when it is released
            if constexpr (PAIR)
                mma_commit_pair_local(smem_addr(drain));
            else
                mma_commit(smem_addr(drain));
            drain_bar(smem_addr(drain), 0, w);
        }
        __syncwarp();
    } else if (warp >= 2 && warp < 2 + kGrEpiWarps) {
        // ------------------------------------------------------ epilogue
        // A warp of quadrant q reads TMEM lanes 32q..32q+31; thread = row.
        constexpr int kCols = BN / 2;            // of this warp
        constexpr int kStep = kCols < 64 ? 32 : 64;
        constexpr int kUnits = kStep / 8;        // of 16 bytes per staged row
        constexpr int kRowsAtOnce = 32 / kUnits; // rows that a warp stores at once
        const int q = warp & 3, half = (warp - 2) / 4;
        uint8_t* stage = staging + (warp - 2) * TS::kUnit;
        // 16 bytes of a staged row: 128-byte rows, units spread over the banks
        auto staged = [&](int r, int k) { return reinterpret_cast<uint4*>(stage + r * 128 + ((k ^ (r & 7)) << 4)); };
        GroupedItems<MODE> items(p, order, worker, workers, TS::kBM);
        GroupedItem it;
        for (int i = 0; items.next(it); ++i) {
            const int row0 = it.tm * TS::kBM + (int)rank * 128 + q * 32;  // this warp's first row, in its group or dB
            const int rows = min(32, (WEIGHT ? p.m : it.cnt) - row0);
            const int n0 = it.tn * BN + half * kCols;                     // and first column
            const bool masked = MODE == GROUPED_ROWS && p.relu_of;
            const uint16_t* mask = nullptr;  // this warp's first row
            if (masked) {
                // its lines are on their way while the products run: 128 bytes per lane and turn
                mask = static_cast<const uint16_t*>(p.relu_of) + (long long)(it.lo + row0) * p.ld_relu;
                constexpr int kLines = kCols < 64 ? 1 : kCols / 64;
                for (int i = lane; i < 32 * kLines; i += 32) {
                    const int r = i / kLines, c = n0 + i % kLines * 64;
                    if (r < rows && c < p.n) asm volatile("prefetch.global.L2 [%0];" ::"l"(mask + (long long)r * p.ld_relu + c));
                }
            }
            Watch whole = w;
            whole.timeout += blocks_of(it) * kGrBlockCycles;
            const bool got = wait_bar(smem_addr(&tfull[i & 1]), (i >> 1) & 1, whole, DEV_TIMEOUT_EPILOGUE + 4);
            if (!__all_sync(0xffffffffu, got)) break;
            tc_fence_after();
            const uint32_t t_row = tmem_base + ((uint32_t)(q * 32) << 16) + (i & 1) * BN + half * kCols;
            auto release = [&]() {  // every column of this buffer is in registers
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR)
                        arrive_on_leader(smem_addr(&tempty[i & 1]));
                    else
                        mbar_arrive(smem_addr(&tempty[i & 1]));
                }
            };
            if (rows <= 0 || n0 >= p.n) {
                release();
                continue;
            }
            uint16_t* out = static_cast<uint16_t*>(p.out) +
                            (WEIGHT ? (long long)it.g * p.out_stride + (long long)row0 * p.ldo
                                    : (long long)(it.lo + row0) * p.ldo);
#pragma unroll 1
            for (int c = 0; c < kCols; c += kStep) {
                const int c0 = n0 + c;
                uint32_t v[kStep / 32][32];
                __syncwarp();
#pragma unroll
                for (int h = 0; h < kStep / 32; ++h) tmem_ld_32x32b_x32(t_row + c + 32 * h, v[h]);
#pragma unroll
                for (int h = 0; h < kStep / 32; ++h) tmem_wait_ld_regs(v[h]);
                if (c + kStep >= kCols) release();
                if (c0 >= p.n) continue;
                float y[kStep];
#pragma unroll
                for (int j = 0; j < kStep; ++j) y[j] = __uint_as_float(v[j / 32][j % 32]);
                if (MODE == GROUPED_ROWS && p.bias) {
                    const uint16_t* b = static_cast<const uint16_t*>(p.bias) + (long long)it.g * p.ld_bias + c0;
#pragma unroll
                    for (int h = 0; h < kStep / 32; ++h) {
                        const float mine = c0 + 32 * h + lane < p.n ? to_f32(b[32 * h + lane], p.bf16) : 0.0f;
#pragma unroll
                        for (int j = 0; j < 32; j += 2)
                            add2(&y[32 * h + j], __shfl_sync(0xffffffffu, mine, j), __shfl_sync(0xffffffffu, mine, j + 1));
                    }
                }
                if (MODE == GROUPED_ROWS && p.relu) {
                    // (a NaN stays one)
#pragma unroll
                    for (int j = 0; j < kStep; ++j) y[j] = y[j] < 0.0f ? 0.0f : y[j];
                }
                __syncwarp();  // the step before has been read
#pragma unroll
                for (int k = 0; k < kUnits; ++k) {
                    const float* f = y + 8 * k;
                    *staged(lane, k) = p.bf16 ? make_uint4(pack2t<true>(f[0], f[1]), pack2t<true>(f[2], f[3]),
                                                           pack2t<true>(f[4], f[5]), pack2t<true>(f[6], f[7]))
                                              : make_uint4(pack2t<false>(f[0], f[1]), pack2t<false>(f[2], f[3]),
                                                           pack2t<false>(f[4], f[5]), pack2t<false>(f[6], f[7]));
                }
                __syncwarp();
                // whole 16-byte units: neighbouring lanes store neighbouring units of a row
                const int k = lane % kUnits, col = c0 + 8 * k;
                constexpr int kTurns = 32 / kRowsAtOnce;
                uint4 z[kTurns];
                if (masked) {
#pragma unroll
                    for (int i = 0; i < kTurns; ++i) {
                        const int r = i * kRowsAtOnce + lane / kUnits;
                        if (r < rows && col < p.n) z[i] = load8(mask + (long long)r * p.ld_relu, col, p.n);
                    }
                }
#pragma unroll
                for (int i = 0; i < kTurns; ++i) {
                    const int r = i * kRowsAtOnce + lane / kUnits;
                    if (r >= rows || col >= p.n) continue;
                    uint4 u = *staged(r, k);
                    if (masked) {
                        uint32_t* word = reinterpret_cast<uint32_t*>(&u);
                        const uint32_t zw[4] = {z[i].x, z[i].y, z[i].z, z[i].w};
                        // above 0: positive, not zero, and no NaN (the largest exponent with a mantissa)
                        const uint32_t inf = p.bf16 ? 0x7F80u : 0x7C00u;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const uint32_t low = zw[x] & 0xFFFFu, high = zw[x] >> 16;
                            word[x] &= (low - 1u < inf ? 0xFFFFu : 0u) | (high - 1u < inf ? 0xFFFF0000u : 0u);
                        }
                    }
                    uint16_t* o = out + (long long)r * p.ldo + col;
                    if (col + 8 <= p.n) {
                        *reinterpret_cast<uint4*>(o) = u;
                    } else {
                        const uint16_t* part = reinterpret_cast<const uint16_t*>(&u);
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            if (col + x < p.n) o[x] = part[x];
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncwarp();
    if (*abort_flag) {
        // copies for phases that were never armed cannot be observed: give
        // them ample time to land
        const long long t0 = clock64();
        while (clock64() - t0 < 2000000) {
        }
    }
    if constexpr (PAIR)
        cluster_sync();  // no CTA leaves while its peer may still signal it
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<CG>(tmem_base, TS::kTmemCols);
    }
}

}  // namespace tg
