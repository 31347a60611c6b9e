// Block operators: which kernels serve a call.
#include "wtconv_block.h"

namespace wtc {

int block_route(const BlockArgs& a, int, int, bool) { return rows_cover(a) ? BLOCK_FUSED : BLOCK_GENERIC; }

size_t block_bwd_workspace_bytes(const BlockArgs& a, int, int) {
    return rows_cover(a) ? rows_bwd_bytes(a) : block_generic_bwd_bytes(a);
}

hipError_t block_fwd_launch(const BlockArgs& a, int h_bf16, int y_bf16, hipStream_t s) {
    return rows_cover(a) ? rows_fwd(a, h_bf16, y_bf16, s) : block_generic_fwd(a, h_bf16, y_bf16, s);
}

hipError_t block_bwd_launch(const BlockArgs& a, int h_bf16, int y_bf16, hipStream_t s) {
    return rows_cover(a) ? rows_bwd(a, h_bf16, y_bf16, s) : block_generic_bwd(a, h_bf16, y_bf16, s);
}

}  // namespace wtc
