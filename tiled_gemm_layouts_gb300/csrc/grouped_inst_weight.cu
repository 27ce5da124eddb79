// Instantiations of the grouped product kernel: GROUPED_WEIGHT.
#include "grouped_launch.cuh"

namespace tg {
template <>
cudaError_t launch_grouped_mode<GROUPED_WEIGHT>(const GroupedParams& p, GroupedTile tile, long long tiles, int sms,
                                                bool chained, cudaStream_t stream) {
    if (tile.pair && tile.bn == 256) return launch_grouped_tile<GROUPED_WEIGHT, 256, true>(p, tiles, sms, chained, stream);
    if (!tile.pair && tile.bn == 128) return launch_grouped_tile<GROUPED_WEIGHT, 128, false>(p, tiles, sms, chained, stream);
    return cudaErrorInvalidValue;
}
}  // namespace tg
