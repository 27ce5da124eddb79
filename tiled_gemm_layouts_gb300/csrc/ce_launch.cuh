// ce_launch.cuh -- the compiled (mode, tile) pairs of the linear cross entropy
// kernel and their launch; each mode is instantiated in its own ce_inst_*.cu
// so that they compile in parallel.
#pragma once

#include <atomic>

#include "ce_kernel.cuh"

namespace tg {

template <int MODE, int BN, bool PAIR, bool DEEP>
cudaError_t launch_ce_kernel(const CeParams& p, int sms, bool chained, cudaStream_t stream) {
    using TS = CeShape<BN, PAIR>;
    auto kern = ce_kernel<MODE, BN, PAIR, DEEP>;
    static std::atomic<unsigned long long> attr_set{0};  // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (!(attr_set.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TS::kCeSmemBytes);
        if (e != cudaSuccess) return e;
        attr_set.fetch_or(bit, std::memory_order_release);
    }
    long long items = 0;
    for (const CeSide& s : p.side)
        items += (long long)s.tiles_m * s.tiles_n * (&s == p.side ? p.splits : 1);
    const long long slots = PAIR ? sms / 2 : sms;
    const int workers = (int)(items < slots ? items : slots);
    cudaLaunchConfig_t lc = {};
    cudaLaunchAttribute attr[2];
    lc.gridDim = dim3(PAIR ? 2 * workers : workers, 1, 1);
    lc.blockDim = dim3(kCeThreads, 1, 1);
    lc.dynamicSmemBytes = TS::kCeSmemBytes;
    lc.stream = stream;
    if (PAIR) {
        attr[lc.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[lc.numAttrs].val.clusterDim.x = 2;
        attr[lc.numAttrs].val.clusterDim.y = 1;
        attr[lc.numAttrs].val.clusterDim.z = 1;
        ++lc.numAttrs;
    }
    if (chained) {
        attr[lc.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[lc.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++lc.numAttrs;
    }
    lc.attrs = attr;
    return cudaLaunchKernelEx(&lc, kern, p);
}

template <int MODE, int BN, bool PAIR>
cudaError_t launch_ce_tile(const CeParams& p, int sms, bool chained, cudaStream_t stream) {
    if constexpr (MODE != CE_PRODUCTS)
        if (p.side[0].num_kb > kCeDepth) return launch_ce_kernel<MODE, BN, PAIR, true>(p, sms, chained, stream);
    return launch_ce_kernel<MODE, BN, PAIR, false>(p, sms, chained, stream);
}

template <int MODE>
cudaError_t launch_ce_mode(const CeParams& p, CeTile tile, int sms, bool chained,
                           cudaStream_t stream);

}  // namespace tg
