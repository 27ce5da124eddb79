// ce_launch.cuh -- the compiled (mode, tile) pairs of the linear cross entropy
// kernel and their launch; each mode is instantiated in its own ce_inst_*.cu
// so that they compile in parallel.
#pragma once

#include <atomic>

#include "ce_kernel.cuh"

namespace tg {

template <int MODE, int BN, bool PAIR>
cudaError_t launch_ce_tile(const CeParams& p, int sms, cudaStream_t stream) {
    using TS = TileShape<BN, PAIR>;
    auto kern = ce_kernel<MODE, BN, PAIR>;
    static std::atomic<unsigned long long> attr_set{0};  // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (!(attr_set.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TS::kSmemBytes);
        if (e != cudaSuccess) return e;
        attr_set.fetch_or(bit, std::memory_order_release);
    }
    const long long items = (long long)p.tiles_m * p.tiles_n * p.splits;
    const long long slots = PAIR ? sms / 2 : sms;
    const int workers = (int)(items < slots ? items : slots);
    cudaLaunchConfig_t lc = {};
    cudaLaunchAttribute attr[1];
    lc.gridDim = dim3(PAIR ? 2 * workers : workers, 1, 1);
    lc.blockDim = dim3(kCeThreads, 1, 1);
    lc.dynamicSmemBytes = TS::kSmemBytes;
    lc.stream = stream;
    if (PAIR) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        lc.attrs = attr;
        lc.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&lc, kern, p);
}

template <int MODE>
cudaError_t launch_ce_mode(const CeParams& p, CeTile tile, int sms, cudaStream_t stream);

}  // namespace tg
