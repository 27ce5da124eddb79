// Instantiations of the linear cross entropy kernel: CE_DH.
#include "ce_launch.cuh"

namespace tg {
template <>
cudaError_t launch_ce_mode<CE_DH>(const CeParams& p, CeTile tile, int sms, cudaStream_t stream) {
    if (tile.pair && tile.bn == 256) return launch_ce_tile<CE_DH, 256, true>(p, sms, stream);
    if (tile.pair && tile.bn == 128) return launch_ce_tile<CE_DH, 128, true>(p, sms, stream);
    if (!tile.pair && tile.bn == 128) return launch_ce_tile<CE_DH, 128, false>(p, sms, stream);
    return cudaErrorInvalidValue;
}
}  // namespace tg
