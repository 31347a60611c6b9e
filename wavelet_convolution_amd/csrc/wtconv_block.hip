// Block operators: which kernels serve a call. Rows (both sides channels last)
// are held in registers by the row kernels up to 16,384 channels, tiles with
// a planar side by the tile kernels from 8 to 2,048 (four pixels at least);
// the others take the generic kernels.
#include "wtconv_block.h"
#include "wtconv_block_tile.h"

namespace wtc {

template <> hipError_t tile_fwd_launch<false, false>(const BlockArgs&, int, int, const TileShape&, hipStream_t);
template <> hipError_t tile_fwd_launch<false, true>(const BlockArgs&, int, int, const TileShape&, hipStream_t);
template <> hipError_t tile_fwd_launch<true, false>(const BlockArgs&, int, int, const TileShape&, hipStream_t);
template <>
hipError_t tile_bwd_launch<false, false>(const BlockArgs&, int, int, const TileShape&, const Partition&, hipStream_t);
template <>
hipError_t tile_bwd_launch<false, true>(const BlockArgs&, int, int, const TileShape&, const Partition&, hipStream_t);
template <>
hipError_t tile_bwd_launch<true, false>(const BlockArgs&, int, int, const TileShape&, const Partition&, hipStream_t);

namespace {

// One tile a workgroup where the card takes them in two rounds, else as many
// workgroups as it holds at once (256 CUs, three wavefronts a SIMD at the
// kernels' registers), each with an even share. Residual backward (layer
// norm, gate per channel, element dropout, residual scale, bf16) 64x96x56x56,
// 1,600 tiles of three wavefronts: 56.8 us at a tile each, 61.5 at 1,024
// workgroups (the card's fill), 76.3 at 1,280; 32x128x128x128, 4,096 tiles of
// four: 163 us at 768 (the fill), 178 at 640, 180 at 1,280, 157 at 2,048 and
// 158 at a tile each, for more partial sums to keep and add.
Partition tile_partition(const BlockArgs& a, const TileShape& t) {
    Partition p{};
    const bool by_sample = a.dg && a.gate_mode == GATE_SAMPLE;
    p.tps = t.tps;
    p.tiles = (long long)a.B * t.tps;
    const long long wgs = 256 * (t.nw > 12 ? 1 : 12 / t.nw);
    p.wgs = (int)(p.tiles <= 2 * wgs ? p.tiles : wgs);
    p.nsum = sum_slots(a).count;
    p.partials = by_sample && p.tps > 1 ? 2 : 0;
    return p;
}

size_t tile_bwd_bytes(const BlockArgs& a, const TileShape& t) {
    const Partition p = tile_partition(a, t);
    return (size_t)p.wgs * (p.nsum + p.partials) * a.C * sizeof(float);
}

// Whether pieces of a plane are no whole 128-byte lines: neighbouring tiles,
// that share the lines between them, then stay on one XCD (32x128x100x100 norm
// forward 32.1 against 37.1 us, 64x384x14x14 residual forward 9.6 against
// 12.7). Where no line is shared that order only spreads the traffic less
// evenly (32x128x128x128 residual forward 89.1 against 81.5 us).
bool shares_lines(const BlockArgs& a, int h_bf16, int y_bf16, const TileShape& t) {
    auto cut = [&](int bf16) { return (size_t)a.HW * (bf16 ? 2 : 4) % 128 != 0 || t.px * (bf16 ? 2 : 4) % 128 != 0; };
    return (!a.h_cl && cut(h_bf16)) || (!a.y_cl && cut(y_bf16));
}

hipError_t tile_fwd(BlockArgs a, int h_bf16, int y_bf16, const TileShape& t, hipStream_t s) {
    if (a.B == 0) return hipSuccess;
    a.near = shares_lines(a, h_bf16, y_bf16, t);
    if (a.h_cl) return tile_fwd_launch<true, false>(a, h_bf16, y_bf16, t, s);
    if (a.y_cl) return tile_fwd_launch<false, true>(a, h_bf16, y_bf16, t, s);
    return tile_fwd_launch<false, false>(a, h_bf16, y_bf16, t, s);
}

hipError_t tile_bwd(BlockArgs a, int h_bf16, int y_bf16, const TileShape& t, hipStream_t s) {
    const Partition p = tile_partition(a, t);
    a.near = shares_lines(a, h_bf16, y_bf16, t);
    if (p.wgs > 0) {
        const hipError_t err = a.h_cl   ? tile_bwd_launch<true, false>(a, h_bf16, y_bf16, t, p, s)
                               : a.y_cl ? tile_bwd_launch<false, true>(a, h_bf16, y_bf16, t, p, s)
                                        : tile_bwd_launch<false, false>(a, h_bf16, y_bf16, t, p, s);
        if (err != hipSuccess) return err;
    }
    return block_finalize(a, p, a.ws, s);
}

}  // namespace

int block_route(const BlockArgs& a, int h_bf16, int y_bf16) {
    return rows_cover(a) || (!(a.h_cl && a.y_cl) && tile_shape(a, h_bf16, y_bf16, true).cl) ? BLOCK_FUSED : BLOCK_GENERIC;
}

size_t block_bwd_workspace_bytes(const BlockArgs& a, int h_bf16, int y_bf16) {
    if (a.h_cl && a.y_cl) return rows_cover(a) ? rows_bwd_bytes(a) : block_generic_bwd_bytes(a);
    const TileShape t = tile_shape(a, h_bf16, y_bf16, true);
    return t.cl ? tile_bwd_bytes(a, t) : block_generic_bwd_bytes(a);
}

hipError_t block_fwd_launch(const BlockArgs& a, int h_bf16, int y_bf16, hipStream_t s) {
    if (rows_cover(a)) return rows_fwd(a, h_bf16, y_bf16, s);
    const TileShape t = a.h_cl && a.y_cl ? TileShape{} : tile_shape(a, h_bf16, y_bf16, false);
    return t.cl ? tile_fwd(a, h_bf16, y_bf16, t, s) : block_generic_fwd(a, h_bf16, y_bf16, s);
}

hipError_t block_bwd_launch(const BlockArgs& a, int h_bf16, int y_bf16, hipStream_t s) {
    if (rows_cover(a)) return rows_bwd(a, h_bf16, y_bf16, s);
    const TileShape t = a.h_cl && a.y_cl ? TileShape{} : tile_shape(a, h_bf16, y_bf16, true);
    return t.cl ? tile_bwd(a, h_bf16, y_bf16, t, s) : block_generic_bwd(a, h_bf16, y_bf16, s);
}

}  // namespace wtc
