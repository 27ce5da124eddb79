// Instantiations of the linear cross entropy kernel: CE_PRODUCTS.
#include "ce_launch.cuh"

namespace tg {
template <>
cudaError_t launch_ce_mode<CE_PRODUCTS>(const CeParams& p, CeTile tile, int sms, bool chained,
                                  cudaStream_t stream) {
    if (tile.pair && tile.bn == 256) return launch_ce_tile<CE_PRODUCTS, 256, true>(p, sms, chained, stream);
    if (tile.pair && tile.bn == 128) return launch_ce_tile<CE_PRODUCTS, 128, true>(p, sms, chained, stream);
    if (!tile.pair && tile.bn == 128) return launch_ce_tile<CE_PRODUCTS, 128, false>(p, sms, chained, stream);
    return cudaErrorInvalidValue;
}
}  // namespace tg
