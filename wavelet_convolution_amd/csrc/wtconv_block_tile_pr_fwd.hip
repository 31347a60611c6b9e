// Tile kernels of the block operators, planar to channels-last rows (forward).
#include "wtconv_block_tile.h"

namespace wtc {

WTC_TILE_FWD(false, true)

}  // namespace wtc
