// grouped_launch.cuh -- the compiled (mode, tile) pairs of the grouped product
// kernel and their launch; each mode is instantiated in its own
// grouped_inst_*.cu so that they compile in parallel.
#pragma once

#include <atomic>

#include "grouped_kernel.cuh"

namespace tg {

template <int MODE, int BN, bool PAIR, bool LIST>
cudaError_t launch_grouped_tile(const GroupedParams& p, long long tiles, int sms,
                                cudaStream_t stream) {
    using TS = GroupedShape<MODE, BN, PAIR, LIST>;
    auto kern = grouped_kernel<MODE, BN, PAIR, LIST>;
    static std::atomic<unsigned long long> attr_set{0};  // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (!(attr_set.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TS::kGrSmemBytes);
        if (e != cudaSuccess) return e;
        attr_set.fetch_or(bit, std::memory_order_release);
    }
    const long long slots = PAIR ? sms / 2 : sms;
    const int workers = (int)(tiles < slots ? tiles : slots);
    cudaLaunchConfig_t lc = {};
    cudaLaunchAttribute attr[1];
    lc.gridDim = dim3(PAIR ? 2 * workers : workers, 1, 1);
    lc.blockDim = dim3(kGrThreads<LIST>, 1, 1);
    lc.dynamicSmemBytes = TS::kGrSmemBytes;
    lc.stream = stream;
    if (PAIR) {
        attr[lc.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[lc.numAttrs].val.clusterDim.x = 2;
        attr[lc.numAttrs].val.clusterDim.y = 1;
        attr[lc.numAttrs].val.clusterDim.z = 1;
        ++lc.numAttrs;
    }
    lc.attrs = attr;
    return cudaLaunchKernelEx(&lc, kern, p);
}

template <int MODE>
cudaError_t launch_grouped_mode(const GroupedParams& p, GroupedTile tile, long long tiles, int sms, cudaStream_t stream);

}  // namespace tg
