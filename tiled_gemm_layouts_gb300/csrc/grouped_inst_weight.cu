// Instantiations of the grouped product kernel: GROUPED_WEIGHT.
#include "grouped_launch.cuh"

namespace tg {
template <>
cudaError_t launch_grouped_mode<GROUPED_WEIGHT>(const GroupedParams& p, GroupedTile tile, long long tiles, int sms, 
                                                cudaStream_t stream) {
    if (tile.bn == 256 && tile.pair && !tile.list)
        return launch_grouped_tile<GROUPED_WEIGHT, 256, true, false>(p, tiles, sms, stream);
    if (tile.bn == 256 && tile.pair && tile.list)
        return launch_grouped_tile<GROUPED_WEIGHT, 256, true, true>(p, tiles, sms, stream);
    if (tile.bn == 128 && !tile.pair && !tile.list)
        return launch_grouped_tile<GROUPED_WEIGHT, 128, false, false>(p, tiles, sms, stream);
    if (tile.bn == 128 && !tile.pair && tile.list)
        return launch_grouped_tile<GROUPED_WEIGHT, 128, false, true>(p, tiles, sms, stream);
    return cudaErrorInvalidValue;
}
}  // namespace tg
