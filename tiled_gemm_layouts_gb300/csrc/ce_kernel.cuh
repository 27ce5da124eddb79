// ce_kernel.cuh -- the tensor-core products of linear cross entropy on
// sm_103a: softmax cross entropy of the logits l = H W^T (H: T x D, W: V x D)
// whose T x V logits never reach memory, and its gradients.
//
//   lse_t = log sum_v exp l_tv          loss_t = lse_t - l_t,target
//   G_tv  = g_t (exp(l_tv - lse_t) - [v = target_t])
//   dH    = G W                         dW = G^T H
//
// The forward pass is one GEMM whose epilogue keeps a running maximum and sum
// of powers of two per accumulator row: in TMEM a tile's row is one lane, so
// the thread that reads it reduces its 128 columns without talking to any
// other, and only 8 bytes per row and half tile leave the SM.  The backward pass
// recomputes the logits piece by piece of the vocabulary (2TVD operations,
// where keeping them would take 2TV or 4TV bytes), writes each piece of G in
// 16 bits, and multiplies it twice.  G is scaled so that its largest possible
// entry is 1 (bf16) or 2^14 (fp16, whose smallest normal number is 2^-14 while
// a probability is about 1/V; rows of light tokens are scaled up further); the
// factors are applied to the fp32 products.
//
// The main loop is that of the GEMM kernel: two TMA producer warps fill a
// ring of 128B-swizzled stages, one thread issues tcgen05.mma into a
// double-buffered fp32 accumulator in TMEM, eight epilogue warps drain it
// while the next tile's products run; tiles of 256 x BN on a CTA pair, or
// 128 x BN on one CTA for few tokens.  Every wait is bounded; on a timeout
// the status word is set, copies and MMAs in flight are drained, TMEM is
// freed and the kernel returns.
//
// What bounds it: at T = 8192, D = 4096, V = 131072 the tensor pipe and the
// power it draws (the loss 4.74 to 5.0 ms, 1760 to 1860 TFLOP/s; at 4096 x
// 2048 x 32768, alone, 2090 TFLOP/s with the tensor pipe 94 % busy).  The
// exponentials run beside the products: 6 % of the special function unit
// there.  At D below about 500 the epilogue shows.  For a few tokens, reading
// W: one token against 131072 x 4096 takes 167 us, 6.4 TB/s.
#pragma once

#include "ce_params.h"
#include "chained.cuh"
#include "gemm_kernel.cuh"

namespace tg {

// Two epilogue warps per TMEM lane quadrant, each with half of a tile's
// columns: one warp's chain of maximum, exponentials and sum leaves its
// scheduler idle half of the time, which shows where a tile's contraction is
// short (D below about 500).
constexpr int kCeEpiWarps = 8;
constexpr int kCeThreads = 32 * (3 + kCeEpiWarps);  // producers (warps 0 and 10), MMA (1), epilogue (2..9)
// Time of an output tile's epilogue in K-blocks: 128 KB of stores at an SM
// pair's share of the memory bandwidth.
constexpr int kCeTileBlocks = 6;
constexpr int kCeBlocksPerStage = 2;              // K-blocks per barrier transaction
constexpr float kLog2e = 1.4426950408889634f;     // logit -> log2 units
// K-blocks that logits sum up in the tensor core's accumulator.  Each
// tcgen05.mma adds 16 products to it and truncates, up to 2^-23 of the partial
// sum each time and always towards zero.  A longer contraction (DEEP) therefore runs
// in parts of this depth; the epilogue warps add the parts in registers, rounded
// to nearest, while the next part's products run.  lse's error against 64 bits
// for random operands, and the loss's time, at 8192 x 4096 x 131072: 2.7e-7,
// 5005 us; one part 1.2e-6, 4960; parts of 8 blocks 1.4e-7, 5057 (and 777 x 1000 x
// 50021 80 us instead of 76).  At D = 16384, where one part loses 5.3e-6, 3.0e-7.
// Reading the accumulator once more per part costs the tensor pipe 1 to 3 %
// (4096 x 2048 x 32768: 314 us, one part 306).
constexpr int kCeDepth = 16;
static_assert(kCeDepth % kCeBlocksPerStage == 0, "whole transactions");

// 2^x; results below the normal range become 0 (for sums of at least 1).
__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^x with gradual underflow, for probabilities that are results themselves.
__device__ __forceinline__ float pow2_gradual(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (a, b) * s + (t, t), as one packed operation.
__device__ __forceinline__ void fma2(float a, float b, float s, float t, float& x, float& y) {
    unsigned long long ab, ss, tt;
    asm("mov.b64 %0, {%1, %2};" : "=l"(ab) : "f"(a), "f"(b));
    asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(s));
    asm("mov.b64 %0, {%1, %1};" : "=l"(tt) : "f"(t));
    asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(ab) : "l"(ss), "l"(tt));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(ab));
}

// Waits for this thread's TMEM loads; the loaded registers pass through, so
// no use of them is scheduled before it.
__device__ __forceinline__ void tmem_wait_ld_regs(uint32_t (&r)[32]) {
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 32; ++j) asm volatile("" : "+r"(r[j]));
}

// Arrives on the leader CTA's barrier once this warp's TMEM loads have
// completed (tcgen05.wait::ld, then the fence before thread synchronisation).
// Nothing else is handed over, so the arrival is relaxed: one that releases
// at cluster scope also waits for the warp's earlier global stores, such as
// the row sums of the tile before, and held the accumulator meanwhile
// (2048 x 128 x 65536: 4700 cycles per tile of 1450 cycles of instructions).
__device__ __forceinline__ void arrive_on_leader(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .b32 ra;\n\t"
        "mapa.shared::cluster.u32 ra, %0, 0;\n\t"
        "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [ra];\n\t}" ::"r"(bar)
        : "memory");
}

// 3-D tensor store and tensor add, shared -> global, fp32.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int c0, int c1,
                                             int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
            reinterpret_cast<uint64_t>(map)),
        "r"(src), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* map, uint32_t src, int c0, int c1,
                                           int c2) {
    asm volatile(
        "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group"
        " [%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
        "r"(src), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// Shared memory of a launch: the ring, and 4 KB of staging per epilogue warp
// (32 rows of 128 bytes: 64 columns of 16 bits or 32 of fp32).  More staging
// at the price of ring slots was slower: 4 slots and 12 KB per warp took 82
// us for 8 x 856 x 54155, 6 slots 75.
template <int BN, bool PAIR>
struct CeShape : TileShape<BN, PAIR> {
    using TS = TileShape<BN, PAIR>;
    static constexpr int kSlots = 6;
    static constexpr int kGroups = kSlots / kCeBlocksPerStage;
    static constexpr int kUnit = 4096;
    static constexpr int kCeSmemBytes =
        1024 + kSlots * TS::kStage + kCeEpiWarps * kUnit + (2 * kGroups + 5) * 8 + 16;
    static_assert(kSlots % kCeBlocksPerStage == 0, "whole groups");
    static_assert(kCeSmemBytes <= TS::kSmemLimit, "shared memory budget");
};

struct CeItem {
    int side, tm, tn, split, kb0, kb1;
};

// The work items of one persistent worker.  `live` shrinks the row tiles or
// the K-blocks to those that hold a row that counts; one is always left, so
// that every output is written (its rows are zeros).
//
// CE_LSE, CE_GRAD: every `workers`-th tile.  CE_PRODUCTS: first every
// `workers`-th (tile, split) of dH; the last round of those leaves some
// workers idle for as long as it takes (at 4096 tokens and columns, 256 tiles
// on 76 pairs: 48 of 76 for a quarter of the time), so these take tiles of dW
// meanwhile; then all share dW's remaining tiles.  The order within a side
// stays a raster, for L2.
template <int MODE>
struct CeItems {
    int tiles_m[2], tiles_n[2], num_kb[2], group_m[2];
    int all_kb, step, stride;
    int at[2], end[2];  // next item of each side, and their numbers
    int tail, tail_at;  // first item of dW's common part, and this worker's next there

    __device__ __forceinline__ CeItems(const CeParams& p, int worker, int workers, int bm)
        : all_kb(p.all_kb), step(workers) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            tiles_m[s] = p.side[s].tiles_m;
            tiles_n[s] = p.side[s].tiles_n;
            num_kb[s] = p.side[s].num_kb;
            group_m[s] = p.side[s].group_m;
        }
        if (p.live) {
            const int n = max(1, *p.live);
            tiles_m[0] = min(tiles_m[0], (n + bm - 1) / bm);
            num_kb[1] = min(num_kb[1], (n + kBK - 1) / kBK);
        }
        end[0] = tiles_m[0] * tiles_n[0] * (MODE == CE_PRODUCTS ? p.splits : 1);
        at[0] = worker;
        if constexpr (MODE == CE_PRODUCTS) {
            const int all = tiles_m[1] * tiles_n[1];
            const int busy = end[0] % workers;  // workers with one more item of dH
            stride = workers - busy;
            const long long rounds =
                busy && all ? max(num_kb[0], kCeTileBlocks) / max(num_kb[1], kCeTileBlocks) : 0;
            tail = (int)min((long long)all, rounds * stride);
            at[1] = worker >= busy ? worker - busy : tail;
            tail_at = tail + worker;
            end[1] = all;
        }
    }
    __device__ __forceinline__ void place(CeItem& it, int i) const {
        const int s = it.side, group = group_m[s] * tiles_n[s];
        const int g = i / group, first = g * group_m[s];
        const int gm = min(tiles_m[s] - first, group_m[s]), r = i - g * group;
        it.tm = first + r % gm;
        it.tn = r / gm;
    }
    __device__ __forceinline__ bool next(CeItem& it) {
        if (at[0] < end[0]) {
            it.side = 0;
            if constexpr (MODE == CE_PRODUCTS) {
                const int tiles = tiles_m[0] * tiles_n[0];
                it.split = at[0] / tiles;
                place(it, at[0] - it.split * tiles);
                it.kb0 = it.split * num_kb[0];
                it.kb1 = min(all_kb, it.kb0 + num_kb[0]);
            } else {
                it.split = 0;
                place(it, at[0]);
                it.kb0 = 0;
                it.kb1 = num_kb[0];
            }
            at[0] += step;
            return true;
        }
        if constexpr (MODE == CE_PRODUCTS) {
            it.side = 1;
            it.split = 0;
            it.kb0 = 0;
            it.kb1 = num_kb[1];
            if (at[1] < tail) {
                place(it, at[1]);
                at[1] += stride;
                return true;
            }
            if (tail_at < end[1]) {
                place(it, tail_at);
                tail_at += step;
                return true;
            }
        }
        return false;
    }
};

// ------------------------------------------------------------ epilogues
//
// Each holds what one thread keeps for its accumulator row and takes the
// tile's columns in chunks of 32, in order.

// The row's running (max, sum): m in log2 units, s the sum of 2^(l - m).
struct CeRowStats {
    float m, s, hit;
    int target;     // column of the target in this launch, or negative

    __device__ __forceinline__ void chunk(const uint32_t (&v)[32], int c0, int cols) {
        float x[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(v[j]);
        chunk(x, c0, cols);
    }
    __device__ __forceinline__ void chunk(float (&x)[32], int c0, int cols) {
        if (c0 >= cols) return;
        if (c0 + 32 > cols) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (c0 + j >= cols) x[j] = -INFINITY;
        }
        const unsigned d = (unsigned)(target - c0);
        if (d < 32u) {
#pragma unroll
            for (int j = 0; j < 32; ++j) hit = d == (unsigned)j ? x[j] * kLog2e : hit;
        }
        float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int j = 4; j < 32; ++j) top[j & 3] = fmaxf(top[j & 3], x[j]);
        const float mc = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * kLog2e;
        const float mn = fmaxf(m, mc);
        const float base = mn == -INFINITY ? 0.0f : mn;  // a row of -inf so far: every term is 0
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            float a, b;
            fma2(x[j], x[j + 1], kLog2e, -base, a, b);
            add2(&sum[j & 2], pow2(a), pow2(b));
        }
        s = s * pow2(m - base) + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
        m = mn;
    }
};

// One kernel for all products.  PAIR: a CTA pair works on 256 x BN tiles.  DEEP:
// logits whose contraction is longer than kCeDepth K-blocks.
template <int MODE, int BN, bool PAIR, bool DEEP>
__global__ void __launch_bounds__(kCeThreads, 1) ce_kernel(const __grid_constant__ CeParams p) {
    using TS = CeShape<BN, PAIR>;
    constexpr bool Q_MN = MODE == CE_PRODUCTS;  // Q's columns contiguous in memory
    constexpr bool BOTH = MODE == CE_PRODUCTS;  // side 1's P (G^T) has its rows contiguous
    constexpr int STAGES = TS::kSlots;
    constexpr int GROUPS = TS::kGroups;
    constexpr int CG = PAIR ? 2 : 1;
    static_assert(!(DEEP && BOTH), "the gradients' products are rounded to 16 bits");
    constexpr uint32_t kQBytes = Q_MN ? (uint32_t)TS::kBStage : (uint32_t)TS::kBNC * 128u;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + STAGES * TS::kAStage;
    uint8_t* staging = sB + STAGES * TS::kBStage;
    uint64_t* full = reinterpret_cast<uint64_t*>(staging + kCeEpiWarps * TS::kUnit);
    uint64_t* empty = full + GROUPS;
    uint64_t* tfull = empty + GROUPS;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
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

    allow_next_kernel();
    if (threadIdx.x == 0) {
        // (a side without work has no maps)
        for (const CeSide& sd : p.side) {
            if (!sd.tiles_m) continue;
            prefetch_tensormap(&sd.map_p);
            prefetch_tensormap(&sd.map_q);
        }
        for (int s = 0; s < GROUPS; ++s) {
            mbar_init(smem_addr(&full[s]), 1);
            mbar_init(smem_addr(&empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(&tfull[b]), 1);
            mbar_init(smem_addr(&tempty[b]), (PAIR ? 2 : 1) * kCeEpiWarps);
        }
        mbar_init(smem_addr(drain), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc<CG>(smem_addr(tmem_slot), TS::kTmemCols);
        tmem_relinquish<CG>();
    }
    tc_fence_before();
    if constexpr (PAIR)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    wait_for_previous_kernel();

    // ------------------------------------------------------ TMA producers
    // Role 1 arms each transaction and loads P, role 2 loads Q into it.
    auto run_producer = [&](auto role) {
        constexpr int ROLE = decltype(role)::value;
        int grp = 0;
        uint32_t phase = 0, armed = 0, armed_parity = 0;
        CeItems<MODE> items(p, worker, workers, TS::kBM);
        CeItem it;
        bool ok = true;
        fence_proxy_async_global();  // H's gathered rows, copies of H and W
        while (ok && items.next(it)) {
            const CeSide& sd = p.side[BOTH ? it.side : 0];
            const bool p_mn = BOTH && it.side == 1;
            const uint32_t stage_tx = (sd.p_bytes + kQBytes) * (PAIR ? 2u : 1u);
            const int m0 = it.tm * TS::kBM + (int)rank * 128;
            const int n0 = it.tn * BN + (int)rank * TS::kBNC;
            const bool whole = Q_MN && n0 + TS::kBNC <= sd.q_whole;
            const int pairs = ROLE == 1 ? sd.p_pairs : !Q_MN || whole ? sd.q_pairs : 0;
            for (int kb = it.kb0; kb < it.kb1; kb += kCeBlocksPerStage) {
                const int n = min(it.kb1 - kb, kCeBlocksPerStage);
                if (!wait_bar(smem_addr(&empty[grp]), phase ^ 1, w, DEV_TIMEOUT_PRODUCER + 1)) {
                    ok = false;
                    break;
                }
                const uint32_t fb_local = smem_addr(&full[grp]);
                if (ROLE == 1 && leader) {
                    mbar_arrive_expect_tx(fb_local, stage_tx * (uint32_t)n);
                    armed |= 1u << grp;
                    armed_parity = (armed_parity & ~(1u << grp)) | (phase << grp);
                }
                const uint32_t fb = PAIR ? mapa_shared(fb_local, 0) : fb_local;
                auto load2 = [&](uint32_t dst, const CUtensorMap* map, int x, int y) {
                    if constexpr (PAIR)
                        tma_load_2d_pair(dst, map, fb, x, y);
                    else
                        tma_load_2d(dst, map, fb, x, y);
                };
                auto load3 = [&](uint32_t dst, const CUtensorMap* map, int x, int y, int z) {
                    if constexpr (PAIR)
                        tma_load_3d_pair(dst, map, fb, x, y, z);
                    else
                        tma_load_3d(dst, map, fb, x, y, z);
                };
                auto load4 = [&](uint32_t dst, const CUtensorMap* map, int y, int z) {
                    if constexpr (PAIR)
                        tma_load_4d_pair(dst, map, fb, 0, 0, y, z);
                    else
                        tma_load_4d(dst, map, fb, 0, 0, y, z);
                };
                const int slot0 = grp * kCeBlocksPerStage;
                const uint32_t dst0 = ROLE == 1 ? smem_addr(sA + slot0 * TS::kAStage)
                                                : smem_addr(sB + slot0 * TS::kBStage);
                constexpr uint32_t kStep = ROLE == 1 ? TS::kAStage : TS::kBStage;
                if (n == 2 && kb + 2 <= pairs) {  // both K-blocks as one box
                    if constexpr (ROLE == 1) {
                        if (p_mn)
                            load4(dst0, &sd.map_p2, m0 >> 6, kb);
                        else
                            load3(dst0, &sd.map_p2, 0, m0, kb);
                    } else if constexpr (Q_MN) {
                        load4(dst0, &sd.map_q2, n0 >> 6, kb);
                    } else {
                        load3(dst0, &sd.map_q2, 0, n0, kb);
                    }
                } else {
                    for (int j = 0; j < n; ++j) {
                        const uint32_t dst = dst0 + j * kStep;
                        const int k0 = (kb + j) * kBK;
                        if constexpr (ROLE == 1) {
                            if (p_mn)
                                load3(dst, &sd.map_p, 0, k0, m0 >> 6);
                            else
                                load2(dst, &sd.map_p, k0, m0);
                        } else if constexpr (Q_MN) {
                            if (whole) {
                                load3(dst, &sd.map_q3, 0, k0, n0 >> 6);
                            } else {
#pragma unroll
                                for (int h = 0; h < TS::kBBoxes; ++h)
                                    load2(dst + h * 8192, &sd.map_q, n0 + 64 * h, k0);
                            }
                        } else {
                            load2(dst, &sd.map_q, k0, n0);
                        }
                    }
                }
                if (++grp == GROUPS) {
                    grp = 0;
                    phase ^= 1;
                }
            }
        }
        if (*abort_flag) {  // no TMA write may land after the CTA exits
            for (int q = 0; q < GROUPS; ++q)
                if (armed & (1u << q)) drain_bar(smem_addr(&full[q]), (armed_parity >> q) & 1, w);
        }
    };

    if (warp == 0 && lane == 0) {
        run_producer(RoleTag<1>{});
    } else if (warp == 2 + kCeEpiWarps && lane == 0) {
        run_producer(RoleTag<2>{});
    } else if (warp == 1 && lane == 0 && leader) {
        // ---------------------------------------------------- MMA issuer
        int grp = 0, i = 0;
        uint32_t phase = 0;
        bool ok = true;
        const uint32_t d_hi = smem_desc_hi_sw128(1024);
        const uint32_t b_lo0 = smem_desc_lo(smem_addr(sB), Q_MN ? 8192u : 16u);
        constexpr uint32_t b_kstep = Q_MN ? (2048u >> 4) : (32u >> 4);
        CeItems<MODE> items(p, worker, workers, TS::kBM);
        CeItem it;
        while (ok && items.next(it)) {
            const bool p_mn = BOTH && it.side == 1;
            const uint32_t idesc = p.side[BOTH ? it.side : 0].idesc;
            const uint32_t a_lo0 = smem_desc_lo(smem_addr(sA), p_mn ? 8192u : 16u);
            const uint32_t a_kstep = p_mn ? (2048u >> 4) : (32u >> 4);
            int start = it.kb0;  // of the part
            do {
                const int end = DEEP ? min(it.kb1, start + kCeDepth) : it.kb1;
                const int buf = i & 1;
                if (!wait_bar(smem_addr(&tempty[buf]), ((i >> 1) & 1) ^ 1, w, DEV_TIMEOUT_MMA + 3)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + buf * BN;
                for (int kb = start; kb < end; kb += kCeBlocksPerStage) {
                    const int n = min(end - kb, kCeBlocksPerStage);
                    if (!wait_bar(smem_addr(&full[grp]), phase, w, DEV_TIMEOUT_MMA + 4)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int j = 0; j < kCeBlocksPerStage; ++j) {
                        if (j >= n) break;
                        const uint32_t slot = (uint32_t)(grp * kCeBlocksPerStage + j);
                        const uint32_t a_lo = a_lo0 + slot * (TS::kAStage >> 4);
                        const uint32_t b_lo = b_lo0 + slot * (TS::kBStage >> 4);
#pragma unroll
                        for (int kk = 0; kk < kBK / kUmmaK; ++kk)
                            mma_f16<CG>(d_tmem, smem_desc_join(a_lo + kk * a_kstep, d_hi),
                                        smem_desc_join(b_lo + kk * b_kstep, d_hi), idesc,
                                        (kb + j != start) || (kk != 0));
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
                if (!ok) break;
                if constexpr (PAIR)
                    mma_commit_pair(smem_addr(&tfull[buf]), 0x3);
                else
                    mma_commit(smem_addr(&tfull[buf]));
                ++i;
                start = end;
            } while (DEEP && start < it.kb1);
        }
        // nothing may still write TMEM when it is released
        if constexpr (PAIR)
            mma_commit_pair_local(smem_addr(drain));
        else
            mma_commit(smem_addr(drain));
        drain_bar(smem_addr(drain), 0, w);
    } else if (warp >= 2 && warp < 2 + kCeEpiWarps) {
        // ------------------------------------------------------ epilogue
        // A warp of quadrant q reads TMEM lanes 32q..32q+31; thread = row.
        constexpr int kChunks = BN / 64;  // of 32 columns, per warp
        static_assert(kChunks % 2 == 0, "chunks are taken in pairs");
        const int q = warp & 3, half = (warp - 2) / 4;
        uint8_t* stage = staging + (warp - 2) * TS::kUnit;
        float alpha = 1.0f;
        if constexpr (MODE == CE_PRODUCTS) alpha = *p.alpha;
        int live = 0;
        if constexpr (MODE == CE_GRAD) live = p.live ? *p.live : p.rows;
        CeItems<MODE> items(p, worker, workers, TS::kBM);
        CeItem it;
        for (int i = 0; items.next(it); ++i) {
            const CeSide& sd = p.side[BOTH ? it.side : 0];
            const int row0 = it.tm * TS::kBM + (int)rank * 128 + q * 32;  // this warp's first row
            const int row = row0 + lane;
            const int n0 = it.tn * BN + half * (BN / 2);  // and first column
            const bool planes = BOTH && it.side == 0;  // fp32 output
            // what the row's epilogue needs, loaded while the products run
            CeRowStats st{-INFINITY, 0.0f, 0.0f, -1};
            float2 rs = make_float2(0.0f, 0.0f);
            int target = -1;
            if constexpr (MODE == CE_LSE) {
                if (row < p.rows) {
                    const long long t = __ldg(p.target + row);
                    if (t >= p.col0 && t < p.col0 + p.cols) st.target = (int)(t - p.col0);
                }
            } else if constexpr (MODE == CE_GRAD) {
                if (row < live) {
                    rs = p.row_scale[row];
                    const long long t = p.row_target[row];
                    if (t >= p.col0 && t < p.col0 + p.cols) target = (int)(t - p.col0);
                }
            }
            // G's rows past the last K-block of dW's contraction are not read
            const bool unused = MODE == CE_GRAD && row0 >= ((max(live, 1) + kBK - 1) & ~(kBK - 1));
            uint32_t t_row;
            auto acquire = [&]() {  // accumulator i, this warp's columns
                const bool got = wait_bar(smem_addr(&tfull[i & 1]), (i >> 1) & 1, w, DEV_TIMEOUT_EPILOGUE + 4);
                tc_fence_after();
                t_row = tmem_base + ((uint32_t)(q * 32) << 16) + (i & 1) * BN + half * (BN / 2);
                return __all_sync(0xffffffffu, got);
            };
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
            uint32_t va[32], vb[32];
            // DEEP: the sum of the contraction's parts before the last
            float sum[DEEP ? kChunks : 1][32];
            auto add_chunk = [&](int c) {
                __syncwarp();
                tmem_ld_32x32b_x32(t_row + c * 32, va);
                tmem_wait_ld_regs(va);
#pragma unroll
                for (int j = 0; j < 32; j += 2)
                    add2(&sum[c][j], __uint_as_float(va[j]), __uint_as_float(va[j + 1]));
            };
            if constexpr (DEEP) {
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[c][j] = 0.0f;
                bool ok = true;
                for (int kb = it.kb0; kb + kCeDepth < it.kb1; kb += kCeDepth, ++i) {
                    ok = acquire();
                    if (!ok) break;
                    if (!unused) {
#pragma unroll
                        for (int c = 0; c < kChunks; ++c) add_chunk(c);
                    }
                    release();
                }
                if (!ok) break;
            }
            if (!acquire()) break;
            if constexpr (MODE == CE_LSE && DEEP) {
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    add_chunk(c);
                    if (c + 1 == kChunks) release();
                    st.chunk(sum[c], n0 + c * 32, p.cols);
                }
            } else if constexpr (MODE == CE_LSE) {
                // the next chunk's TMEM load runs beside this chunk's arithmetic
                __syncwarp();
                tmem_ld_32x32b_x32(t_row, va);
#pragma unroll 1
                for (int c = 0; c < kChunks; c += 2) {
                    tmem_wait_ld_regs(va);
                    __syncwarp();
                    tmem_ld_32x32b_x32(t_row + (c + 1) * 32, vb);
                    st.chunk(va, n0 + c * 32, p.cols);
                    tmem_wait_ld_regs(vb);
                    if (c + 2 < kChunks) {
                        __syncwarp();
                        tmem_ld_32x32b_x32(t_row + (c + 2) * 32, va);
                    } else {
                        release();
                    }
                    st.chunk(vb, n0 + (c + 1) * 32, p.cols);
                }
            } else {
                // 64 columns at a time: staged in swizzled shared memory and
                // written with one tensor store, clipped by the map.  The
                // fence and the store's issue are most of a step's latency
                // (500 of 1150 cycles at 32 columns), so steps are wide.
                auto logits_to_gradient = [&](float (&y)[32], int c0) {
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        fma2(y[j], y[j + 1], kLog2e, -rs.x, y[j], y[j + 1]);
                        y[j] = pow2_gradual(y[j]);
                        y[j + 1] = pow2_gradual(y[j + 1]);
                    }
                    const unsigned d = (unsigned)(target - c0);
                    if (__any_sync(0xffffffffu, d < 32u)) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (d == (unsigned)j) y[j] -= 1.0f;
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 2) mul2(y + j, rs.y);
                    // no token: H's row is zeros, but W may hold infinities
                    if (row0 + 32 > live) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (row >= live) y[j] = 0.0f;
                    }
                    if (c0 + 32 > p.cols) {  // the piece's padding columns hold zeros
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (c0 + j >= p.cols) y[j] = 0.0f;
                    }
                };
                // 16 bytes of this lane's staged row
                auto staged = [&](int k) {
                    return reinterpret_cast<uint4*>(stage + lane * 128 + ((k ^ (lane & 7)) << 4));
                };
                auto stage_free = [&]() {
                    if (lane == 0) bulk_wait_group_read<0>();
                    __syncwarp();
                };
                auto stage_full = [&]() {
                    fence_proxy_async_shared();
                    __syncwarp();
                };
                if (unused) {
                    release();
                    continue;
                }
                // the accumulator's columns from chunk c, and the next chunk's
                auto step = [&](int c, float (&ya)[32], float (&yb)[32]) {
                    const int c0 = n0 + c * 32;
                    if (planes) {
                        // 32 fp32 columns per store
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            stage_free();
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const float* y = (h ? yb : ya) + 4 * k;
                                *staged(k) = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]),
                                                        __float_as_uint(y[2]), __float_as_uint(y[3]));
                            }
                            stage_full();
                            if (lane == 0) {
                                const int c1 = c0 + 32 * h;
                                if (row0 < sd.out_rows && c1 < sd.out_cols) {
                                    if (p.accumulate)
                                        tma_add_3d(&sd.map_c, smem_addr(stage), c1, row0, it.split);
                                    else
                                        tma_store_3d(&sd.map_c, smem_addr(stage), c1, row0, it.split);
                                }
                                bulk_commit_group();
                            }
                        }
                        return;
                    }
                    if constexpr (MODE == CE_GRAD) {
                        logits_to_gradient(ya, c0);
                        logits_to_gradient(yb, c0 + 32);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            mul2(ya + j, alpha);
                            mul2(yb + j, alpha);
                        }
                    }
                    stage_free();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float* y = (k < 4 ? ya : yb) + 8 * (k & 3);
                        *staged(k) = p.bf16 ? make_uint4(pack2t<true>(y[0], y[1]), pack2t<true>(y[2], y[3]),
                                                         pack2t<true>(y[4], y[5]), pack2t<true>(y[6], y[7]))
                                            : make_uint4(pack2t<false>(y[0], y[1]), pack2t<false>(y[2], y[3]),
                                                         pack2t<false>(y[4], y[5]), pack2t<false>(y[6], y[7]));
                    }
                    stage_full();
                    if (lane == 0) {
                        if constexpr (BOTH) {
                            // dW is not read again: its lines leave L2 first
                            if (row0 < sd.out_rows && c0 < p.n_tma)
                                tma_store_2d_hint(&sd.map_c, smem_addr(stage), c0, row0,
                                                  l2_policy_evict_first());
                        } else {
                            tma_store_2d(&sd.map_c, smem_addr(stage), c0, row0);
                        }
                        bulk_commit_group();
                    }
                    // columns the map cannot hold (all of them for an unaligned
                    // dW): half a row of the step per store, lane = column.  The
                    // sectors that two stores share cost what they cost: 8 x 2001
                    // x 40001 takes 108 us here where aligned rows take 60, and
                    // 16-byte windows aligned in dW, 4 rows per store, took 125.
                    if (BOTH && c0 + 64 > p.n_tma && c0 < sd.out_cols) {
                        uint16_t* o = static_cast<uint16_t*>(p.out) + (long long)row0 * p.ldo + c0;
                        const int rows = min(32, sd.out_rows - row0);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int x = 32 * h + lane;
                            if (c0 + x < p.n_tma || c0 + x >= sd.out_cols) continue;
#pragma unroll 8
                            for (int r = 0; r < rows; ++r)
                                o[(long long)r * p.ldo + x] = *reinterpret_cast<const uint16_t*>(
                                    stage + r * 128 + (((x >> 3) ^ (r & 7)) << 4) + (x & 7) * 2);
                        }
                        __syncwarp();
                    }
                };
                if constexpr (DEEP) {
#pragma unroll
                    for (int c = 0; c < kChunks; c += 2) {
                        add_chunk(c);
                        add_chunk(c + 1);
                        if (c + 2 == kChunks) release();
                        step(c, sum[c], sum[c + 1]);
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < kChunks; c += 2) {
                        __syncwarp();
                        tmem_ld_32x32b_x32(t_row + c * 32, va);
                        tmem_ld_32x32b_x32(t_row + (c + 1) * 32, vb);
                        tmem_wait_ld_regs(va);
                        tmem_wait_ld_regs(vb);
                        if (c + 2 == kChunks) release();
                        float ya[32], yb[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            ya[j] = __uint_as_float(va[j]);
                            yb[j] = __uint_as_float(vb[j]);
                        }
                        step(c, ya, yb);
                    }
                }
            }
            if constexpr (MODE == CE_LSE) {
                if (row < p.rows) {
                    p.part[((long long)row * sd.tiles_n + it.tn) * 2 + half] = make_float2(st.m, st.s);
                    const int t = st.target - n0;
                    if (t >= 0 && t < BN / 2) p.hit[row] = st.hit;
                }
            }
        }
        if (lane == 0) bulk_wait_group<0>();  // every output chunk has reached global memory
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
