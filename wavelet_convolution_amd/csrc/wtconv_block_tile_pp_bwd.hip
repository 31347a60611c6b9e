// Tile kernels of the block operators, planar to planar (backward).
#include "wtconv_block_tile.h"

namespace wtc {

WTC_TILE_BWD(false, false)

}  // namespace wtc
