// ring.cuh -- rows of 16-bit elements, at any address, through a ring of bulk
// copies in shared memory.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "gemm_params.h"
#include "ptx.cuh"
#include "stage.cuh"

namespace tg {

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// Bounded wait for a stage; on a timeout the status word is set, and copies
// in flight get ample time to land before the block may end.
__device__ __forceinline__ bool stage_ready(uint32_t bar, uint32_t parity, long long timeout_cycles,
                                            int* status) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait_suspend(bar, parity, 200000)) {
        if (clock64() - t0 > timeout_cycles) {
            atomicCAS(status, 0, DEV_TIMEOUT_PRODUCER + 2);
            const long long t1 = clock64();
            while (clock64() - t1 < 2000000) {
            }
            return false;
        }
    }
    return true;
}

// The bulk copy of `n` elements into a stage: the aligned 16-byte units around
// them.  Units that reach past the operand's end are left out, and their part
// of the elements is stored by this thread; it arrives on the stage's barrier
// afterwards, which hands them over.
struct RowCopy {
    const uint8_t* src;
    uint32_t bytes;
};
__device__ __forceinline__ RowCopy row_copy(uint8_t* dst, const uint16_t* row, const uint16_t* end, int n) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row), from = at & ~uintptr_t(15);
    const uint32_t lead = (uint32_t)(at - from), need = lead + (uint32_t)n * 2;
    uint32_t bytes = (need + 15) & ~15u;
    if (from + bytes > reinterpret_cast<uintptr_t>(end)) {
        bytes = need & ~15u;
        for (uint32_t k = max(bytes, lead); k < need; k += 2)
            *reinterpret_cast<uint16_t*>(dst + k) = row[(k - lead) / 2];
    }
    return {reinterpret_cast<const uint8_t*>(from), bytes};
}

// 8 elements from `off` elements into unit `k` of a stage.
__device__ __forceinline__ uint4 window(const uint8_t* stage, int k, int off) {
    const uint4* v = reinterpret_cast<const uint4*>(stage) + k + (off >> 3);
    const int s = off & 7;
    uint4 a = v[0];
    if (s) a = funnel(a, v[1], s);
    return a;
}

}  // namespace tg
