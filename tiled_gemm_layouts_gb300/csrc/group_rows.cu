// group_rows.cu -- rows grouped by an index: a stable counting sort
// (tg_group_rows).
//
//   place[i] = (rows of smaller groups) + (earlier rows of the same group)
//
// Blocks take 2048 consecutive rows, a warp 256 of them.  Rows of one group
// within 32 are ranked by a match across the warp; a warp's counts per group
// live in shared memory and become, by a sum over the warps before it, the
// places its rows start from.  What the blocks before hold is counted by a first
// kernel, block by block, into the workspace; every block of the second adds
// those counts up for itself (64 blocks x 256 groups are 64 KB, out of L2).
// (More blocks than 64 have a kernel between the two add them up, so that the
// work stays proportional to the rows.)  So a row's place depends on nothing but
// its index and number, whatever order the blocks run in.  Bound by latency: two short kernels, the second's
// launch hidden behind the first (one kernel where one block holds all rows).
#include <cuda_runtime.h>

#include <cstring>

#include "../../include/tilegemm.h"
#include "chained.cuh"
#include "host_common.h"

namespace tg {
namespace {

constexpr int kGroupWarps = 8;
constexpr int kGroupThreads = 32 * kGroupWarps;
constexpr int kRowsPerWarp = 256;
constexpr int kRowsPerBlock = kGroupWarps * kRowsPerWarp;
constexpr int kMaxGroups = 4096;
constexpr int kBlocksAdded = 64;  // that each block adds up for itself

// Shared memory of place_kernel.
constexpr size_t place_bytes(int64_t G) { return (size_t)(2 * G + 1) * 4 + (size_t)kGroupWarps * G * 2; }

// counts[block][g]: rows of group g among the block's
__global__ void __launch_bounds__(kGroupThreads) count_kernel(const int* index, int R, int G, int* counts) {
    extern __shared__ int shared_counts[];
    allow_next_kernel();
    for (int g = threadIdx.x; g < G; g += kGroupThreads) shared_counts[g] = 0;
    __syncthreads();
    const int first = blockIdx.x * kRowsPerBlock;
    for (int i = first + threadIdx.x; i < min(R, first + kRowsPerBlock); i += kGroupThreads) {
        const int g = index[i];
        if (g >= 0 && g < G) atomicAdd(&shared_counts[g], 1);
    }
    __syncthreads();
    for (int g = threadIdx.x; g < G; g += kGroupThreads) counts[(long long)blockIdx.x * G + g] = shared_counts[g];
}

// counts[block][g] to the rows of the blocks before; all[g]: of all of them
__global__ void __launch_bounds__(kGroupThreads) scan_kernel(int blocks, int G, int* counts, int* all) {
    allow_next_kernel();
    const int g = blockIdx.x * kGroupThreads + threadIdx.x;
    if (g >= G) return;
    wait_for_previous_kernel();
    int run = 0;
    for (int b0 = 0; b0 < blocks; b0 += 32) {
        int n[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) n[j] = b0 + j < blocks ? counts[(long long)(b0 + j) * G + g] : 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (b0 + j < blocks) counts[(long long)(b0 + j) * G + g] = run;
            run += n[j];
        }
    }
    all[g] = run;
}

// shared memory: start[G + 1] and earlier[G] ints, then counts of 16 bits [kGroupWarps][G]
__global__ void __launch_bounds__(kGroupThreads) place_kernel(const int* index, int R, int G, const int* counts,
                                                              const int* totals, int* offset, int* row, int* place) {
    extern __shared__ int start[];
    __shared__ int warp_total[kGroupWarps];
    int* earlier = start + G + 1;  // rows of each group in the blocks before
    uint16_t* mine = reinterpret_cast<uint16_t*>(earlier + G);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = blockIdx.x * kRowsPerBlock + warp * kRowsPerWarp;
    for (int g = threadIdx.x; g < kGroupWarps * G; g += kGroupThreads) mine[g] = 0;
    // this warp's rows
    constexpr int kSteps = kRowsPerWarp / 32;
    int of[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int i = first + s * 32 + lane;
        const int g = i < R ? index[i] : -1;
        of[s] = g >= 0 && g < G ? g : -1;
    }
    __syncthreads();
    uint16_t* own = mine + warp * G;
    // lanes whose row is of the same group, from one ballot per bit of its number
    const int bits = 32 - __clz(G);  // (so none of -1's lanes agrees with another's)
    auto peers_of = [&](int g) {
        unsigned peers = 0xffffffffu;
        for (int b = 0; b < bits; ++b) {
            const unsigned set = __ballot_sync(0xffffffffu, g >> b & 1);
            peers &= g >> b & 1 ? set : ~set;
        }
        return peers;
    };
    // its rows' ranks among the warp's of their groups, and the warp's counts
    const unsigned lower = (1u << lane) - 1u;
    int rank[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const unsigned peers = peers_of(of[s]);
        const int before = of[s] >= 0 ? own[of[s]] : 0;
        rank[s] = before + __popc(peers & lower);
        __syncwarp();
        if (of[s] >= 0 && (peers & lower) == 0) own[of[s]] = (uint16_t)(before + __popc(peers));
        __syncwarp();
    }
    __syncthreads();
    wait_for_previous_kernel();
    // start[g + 1]: rows of group g in all blocks; own counts: rows of the warps before.
    // A thread takes the same groups below, so that it may keep what it adds up.
    for (int g = threadIdx.x; g < G; g += kGroupThreads) {
        int before = 0;
        for (int w = 0; w < kGroupWarps; ++w) {
            const int n = mine[w * G + g];
            mine[w * G + g] = (uint16_t)before;
            before += n;
        }
        int all = before;
        if (totals) {
            all = totals[g];
            earlier[g] = counts[(long long)blockIdx.x * G + g];
        } else if (counts) {  // the blocks', 32 loads in flight
            all = 0;
            int ahead = 0;
            for (int b0 = 0; b0 < (int)gridDim.x; b0 += 32) {
                int n[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) n[j] = b0 + j < (int)gridDim.x ? counts[(long long)(b0 + j) * G + g] : 0;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    all += n[j];
                    if (b0 + j < (int)blockIdx.x) ahead += n[j];
                }
            }
            earlier[g] = ahead;
        }
        start[g + 1] = all;
    }
    if (threadIdx.x == 0) start[0] = 0;
    __syncthreads();
    // running sums: a thread takes consecutive groups
    const int per = (G + kGroupThreads - 1) / kGroupThreads;
    const int lo = min(G, (int)threadIdx.x * per), hi = min(G, lo + per);
    int sum = 0;
    for (int g = lo; g < hi; ++g) sum += start[g + 1];
    int run = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, run, d);
        if (lane >= d) run += o;
    }
    if (lane == 31) warp_total[warp] = run;
    __syncthreads();
    run -= sum;
    for (int w = 0; w < warp; ++w) run += warp_total[w];
    for (int g = lo; g < hi; ++g) {
        run += start[g + 1];
        start[g + 1] = run;
    }
    __syncthreads();
    const int total = start[G];
    if (blockIdx.x == 0)
        for (int g = threadIdx.x; g <= G; g += kGroupThreads) offset[g] = start[g];
    __syncthreads();
    // the places this block's rows start from
    if (counts) {
        for (int g = threadIdx.x; g < G; g += kGroupThreads) start[g] += earlier[g];
        __syncthreads();
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int i = first + s * 32 + lane, g = of[s];
        const int at = g >= 0 ? start[g] + own[g] + rank[s] : -1;
        if (i < R) {
            if (at >= 0) row[at] = i;
            if (place) place[i] = at;
            // the places behind the last group's, one of this thread's for each of its rows
            if (i >= total) row[i] = -1;
        }
    }
}

int check_counts(int64_t R, int64_t G) {
    return R <= 0 || G <= 0 || R > kMaxSize || G > kMaxGroups ? TG_ERR_INVALID_ARG : TG_OK;
}

int64_t blocks_of(int64_t R) { return (R + kRowsPerBlock - 1) / kRowsPerBlock; }

}  // namespace
}  // namespace tg

using namespace tg;

extern "C" int tg_group_rows_workspace_size(int64_t R, int64_t G, size_t* bytes) {
    const int rc = check_counts(R, G);
    if (rc) return rc;
    if (!bytes) return TG_ERR_INVALID_ARG;
    const int64_t blocks = blocks_of(R);
    *bytes = blocks > 1 ? (size_t)(blocks + (blocks > kBlocksAdded)) * (size_t)G * sizeof(int) : 0;
    return TG_OK;
}

extern "C" int tg_group_rows(int64_t R, int64_t G, const int32_t* index, int32_t* offset, int32_t* row,
                             int32_t* place, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    int rc = check_counts(R, G);
    if (rc) return rc;
    size_t need = 0;
    tg_group_rows_workspace_size(R, G, &need);
    if (!index || !offset || !row || (need && !workspace)) return TG_ERR_INVALID_ARG;
    auto off = [](const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; };
    if (off(index, 4) || off(offset, 4) || off(row, 4) || off(place, 4) || (need && off(workspace, 256)))
        return TG_ERR_ALIGN;
    if (workspace_bytes < need) return TG_ERR_BUFFER;
    const void* ptrs[5] = {offset, row, place, need ? workspace : nullptr, index};
    const Span spans[5] = {span_bytes(offset, (u128)(G + 1) * 4), span_bytes(row, (u128)R * 4),
                           span_bytes(place, (u128)R * 4), span_bytes(ptrs[3], need), span_bytes(index, (u128)R * 4)};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 5; ++j)
            if (intersects(spans[i], spans[j])) return TG_ERR_OVERLAP;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    load_driver_entry_points();  // the allocation-range query of check_pointer
    PointerChecks check{dev};
    for (int i = 0; i < 5; ++i)
        if ((rc = check(ptrs[i], spans[i]))) return rc;
    const unsigned blocks = (unsigned)blocks_of(R);
    int* counts = need ? static_cast<int*>(workspace) : nullptr;
    const size_t shared = place_bytes(G);
    cudaError_t e = cudaSuccess;
    if (shared > 48 * 1024)  // (the most of all calls: another thread's may be on its way)
        e = cudaFuncSetAttribute(place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)place_bytes(kMaxGroups));
    if (e == cudaSuccess && counts) {
        count_kernel<<<blocks, kGroupThreads, (size_t)G * 4, stream>>>(index, (int)R, (int)G, counts);
        e = cudaGetLastError();
    }
    int* totals = blocks > (unsigned)kBlocksAdded ? counts + (size_t)blocks * (size_t)G : nullptr;
    if (e == cudaSuccess && totals)
        e = launch_chained(scan_kernel, dim3((unsigned)((G + kGroupThreads - 1) / kGroupThreads)), kGroupThreads, stream, (int)blocks,
                           (int)G, counts, totals);
    if (e == cudaSuccess) {
        cudaLaunchConfig_t lc = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        lc.gridDim = dim3(blocks, 1, 1);
        lc.blockDim = dim3(kGroupThreads, 1, 1);
        lc.dynamicSmemBytes = shared;
        lc.stream = stream;
        lc.attrs = attr;
        lc.numAttrs = counts ? 1 : 0;
        e = cudaLaunchKernelEx(&lc, place_kernel, (const int*)index, (int)R, (int)G, (const int*)counts,
                               (const int*)totals, (int*)offset, (int*)row, (int*)place);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return TG_ERR_CUDA;
    }
    return TG_OK;
}
