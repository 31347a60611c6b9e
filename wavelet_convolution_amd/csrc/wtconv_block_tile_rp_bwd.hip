// Tile kernels of the block operators, channels-last rows to planar (backward).
#include "wtconv_block_tile.h"

namespace wtc {

WTC_TILE_BWD(true, false)

}  // namespace wtc
