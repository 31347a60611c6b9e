// The block operators: channel norm, block residual and counter dropout.
//
// A row is the C channels of one pixel (b, p), p < HW. With h the norm's
// input (or the block's output) and y the result (for the residual, x and y
// are the residual stream):
//   z = (h - mean) r, r = 1 / sqrt(var + eps)   (layer; rms: mean = 0, var = mean of h^2; none: z = h)
//   v = z w + b,  t = D(v),  y = s x + g t
// and backwards, for dy:
//   dx = s dy, ds = sum dy x, dg = sum dy t, dv = D'(g dy), dw = sum dv z, db = sum dv, u = dv w,
//   dh = r (u - mean(u) - z mean(u z))          (rms: without mean(u); none: dh = dv)
// The norm alone is the case without x, g and D.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "wtconv_device.h"

namespace wtc {

enum { NORM_NONE = 0, NORM_LAYER = 1, NORM_RMS = 2 };
enum { GATE_NONE = 0, GATE_CHANNEL = 1, GATE_SAMPLE = 2 };
enum { DROP_NONE = 0, DROP_ELEMENT = 1, DROP_SAMPLE = 2 };

// Channels that share one generator call: 16 of its 128 bits each.
constexpr int CG = 8;

// What a call has and wants, as bits: the backward kernels test them inside
// their loop (a test of a bit there is two scalar instructions; conditions
// kept over the loop were most of its scalar registers).
enum : uint32_t {
    HAS_W = 1, HAS_GATE = 2, HAS_XS = 4, WANT_DX = 8, WANT_DH = 16, WANT_DXS = 32, LAYER = 64, RMS = 128,
    BY_SAMPLE = 256, DROPS_SAMPLES = 512, EACH_ROW = 1024
};

struct BlockArgs {
    const void* h;
    const void* x;      // residual stream in (null: none)
    void* y;            // forward result
    const void* dy;
    void* dx;           // null: not wanted
    void* dh;           // null: not wanted
    const float *w, *b, *gate, *xs;   // null: 1, 0, 1, 1
    const unsigned long long* rng;    // seed, offset
    float *dw, *db, *dg, *dxs;        // null: not wanted
    float* ws;
    int B, C, HW;
    int h_cl, y_cl;     // channels last
    int norm, gate_mode, drop;
    float eps;
    float inv_c;        // 1 / C
    uint32_t thr;       // an element is kept when its 16 bits are >= thr
    float keep;         // 65536 / (65536 - thr); 0 where thr = 65536
    uint32_t site;
    uint32_t flags;     // of the backward kernels, set at their launch
    uint32_t near;      // neighbouring tiles share cache lines: keep them on one XCD
};

// The sums over rows that the parameter gradients need. Each workgroup of a
// backward kernel adds over a contiguous range of tiles (a tile: some rows
// of one sample; the ranges differ by one tile at most, evenly over the
// workgroups, so that the CUs' shares differ little), and leaves its sums in
// its slot of the workspace; a second
// stage adds the slots in order, so results do not depend on timing. With a
// gate per sample, a workgroup writes the gate gradient of a sample whose
// tiles are all its own, and leaves at most two partial sums (its first and
// its last sample) for the second stage.
struct Partition {
    long long tiles;    // all tiles
    long long tps;      // tiles per sample (samples count only with a gate per sample: else one)
    int wgs;            // workgroups: at most one a tile; each kernel's rule is at its partition
    int nsum;           // channel sums a slot holds
    int partials;       // 0, or 2: partial gate gradients per slot
    __host__ __device__ long long begin(long long wg) const { return wg * tiles / wgs; }
    __host__ __device__ long long owner(long long tile) const { return ((tile + 1) * wgs - 1) / tiles; }
};

// Places of the channel sums in a slot; -1: not wanted.
struct SumSlots {
    int dw, db, dg, dxs, count;
};
inline SumSlots sum_slots(const BlockArgs& a) {
    SumSlots s{-1, -1, -1, -1, 0};
    if (a.dw) s.dw = s.count++;
    if (a.db) s.db = s.count++;
    if (a.dg && a.gate_mode == GATE_CHANNEL) s.dg = s.count++;
    if (a.dxs) s.dxs = s.count++;
    return s;
}

inline uint32_t block_flags(const BlockArgs& a) {
    const bool sample = a.gate_mode == GATE_SAMPLE;
    return (a.w ? HAS_W : 0) | (a.gate ? HAS_GATE : 0) | (a.xs ? HAS_XS : 0) | (a.dx ? WANT_DX : 0) |
           (a.dh ? WANT_DH : 0) | (a.dxs ? WANT_DXS : 0) | (a.norm == NORM_LAYER ? LAYER : 0) |
           (a.norm == NORM_RMS ? RMS : 0) | (sample && a.HW > 1 ? BY_SAMPLE : 0) |
           (a.drop == DROP_SAMPLE ? DROPS_SAMPLES : 0) | (sample && a.HW == 1 ? EACH_ROW : 0);
}

// A backward call that is more than a norm's.
inline bool block_residual(const BlockArgs& a) {
    return a.gate || a.xs || a.dx || a.dxs || a.drop != DROP_NONE;
}

// How a call is served: by which kernels, and with how much workspace.
enum { BLOCK_GENERIC = 0, BLOCK_FUSED = 1 };
int block_route(const BlockArgs& a, int h_bf16, int y_bf16);
size_t block_bwd_workspace_bytes(const BlockArgs& a, int h_bf16, int y_bf16);
hipError_t block_fwd_launch(const BlockArgs& a, int h_bf16, int y_bf16, hipStream_t s);
hipError_t block_bwd_launch(const BlockArgs& a, int h_bf16, int y_bf16, hipStream_t s);
hipError_t dropout_launch(const BlockArgs& a, int bf16, hipStream_t s);

// generic kernels (any size and layout)
size_t block_generic_bwd_bytes(const BlockArgs& a);
hipError_t block_generic_fwd(const BlockArgs& a, int h_bf16, int y_bf16, hipStream_t s);
hipError_t block_generic_bwd(const BlockArgs& a, int h_bf16, int y_bf16, hipStream_t s);

// rows in registers (both sides channels last)
bool rows_cover(const BlockArgs& a);
size_t rows_bwd_bytes(const BlockArgs& a);
hipError_t rows_fwd(const BlockArgs& a, int h_bf16, int y_bf16, hipStream_t s);
hipError_t rows_bwd(const BlockArgs& a, int h_bf16, int y_bf16, hipStream_t s);

// second stage
hipError_t block_finalize(const BlockArgs& a, const Partition& p, const float* ws, hipStream_t s);

}  // namespace wtc
