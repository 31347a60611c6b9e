// Tile kernels of the block operators, planar to planar (forward).
#include "wtconv_block_tile.h"

namespace wtc {

WTC_TILE_FWD(false, false)

}  // namespace wtc
