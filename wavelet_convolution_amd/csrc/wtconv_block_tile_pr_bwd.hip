// Tile kernels of the block operators, planar to channels-last rows (backward).
#include "wtconv_block_tile.h"

namespace wtc {

WTC_TILE_BWD(false, true)

}  // namespace wtc
