// Instantiations of the grouped product kernel: GROUPED_ROWS.
#include "grouped_launch.cuh"

namespace tg {
template <>
cudaError_t launch_grouped_mode<GROUPED_ROWS>(const GroupedParams& p, GroupedTile tile, long long tiles, int sms, 
                                              cudaStream_t stream) {
    if (tile.bn == 256 && tile.pair && !tile.list)
        return launch_grouped_tile<GROUPED_ROWS, 256, true, false>(p, tiles, sms, stream);
    if (tile.bn == 256 && tile.pair && tile.list)
        return launch_grouped_tile<GROUPED_ROWS, 256, true, true>(p, tiles, sms, stream);
    if (tile.bn == 128 && !tile.pair && !tile.list)
        return launch_grouped_tile<GROUPED_ROWS, 128, false, false>(p, tiles, sms, stream);
    if (tile.bn == 128 && !tile.pair && tile.list)
        return launch_grouped_tile<GROUPED_ROWS, 128, false, true>(p, tiles, sms, stream);
    if (tile.bn == 64 && !tile.pair && !tile.list)
        return launch_grouped_tile<GROUPED_ROWS, 64, false, false>(p, tiles, sms, stream);
    if (tile.bn == 64 && !tile.pair && tile.list)
        return launch_grouped_tile<GROUPED_ROWS, 64, false, true>(p, tiles, sms, stream);
    return cudaErrorInvalidValue;
}
}  // namespace tg
