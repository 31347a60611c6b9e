// Tile kernels of the block operators, channels-last rows to planar (forward).
#include "wtconv_block_tile.h"

namespace wtc {

WTC_TILE_FWD(true, false)

}  // namespace wtc
