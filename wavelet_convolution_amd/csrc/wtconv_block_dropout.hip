// Counter dropout: y = keep ? x * 65536 / (65536 - thr) : 0, the mask computed
// from (seed, offset, site, element) and never stored; the backward pass is
// the same call on dy.
#include "wtconv_block_device.h"

namespace wtc {
namespace {

constexpr int T = 256;

// A thread takes the eight channels of one group in one row: one generator
// call, whatever the layout.
template <typename X>
__global__ __launch_bounds__(T) void k_dropout_generic(BlockArgs a) {
    const X* h = (const X*)a.h;
    X* y = (X*)a.y;
    const long long G = cdiv(a.C, CG), rows = (long long)a.B * a.HW, items = rows * G;
    for (long long n = (long long)blockIdx.x * T + threadIdx.x; n < items; n += (long long)gridDim.x * T) {
        // neighbouring threads: channels of a row in rows, pixels of a plane in planes
        long long row, g;
        if (a.h_cl) {
            row = n / G;
            g = n - row * G;
        } else {
            const long long bg = n / a.HW, p = n - bg * a.HW, b = bg / G;
            g = bg - b * G;
            row = b * a.HW + p;
        }
        const long long b = row / a.HW;
        const size_t step = a.h_cl ? 1 : (size_t)a.HW;
        const size_t at = (a.h_cl ? (size_t)row * a.C : (size_t)b * a.C * a.HW + (row - b * a.HW)) + g * CG * step;
        uint32_t m;
        if (a.drop == DROP_SAMPLE) {
            m = sample_kept(a, (int)b) ? 0u : ALL_DROPPED;
        } else {
            const Philox gen(a.rng, a.site);
            m = drop_bits(gen((uint32_t)row * (uint32_t)G + (uint32_t)g), a.thr);
        }
        for (int i = 0; i < CG && g * CG + i < a.C; ++i)
            y[at + i * step] = narrow_to<X>(kept(widen(h[at + i * step]) * a.keep, m, i));
    }
}

}  // namespace

hipError_t dropout_launch(const BlockArgs& a, int bf16, hipStream_t s) {
    const long long items = (long long)a.B * a.HW * cdiv(a.C, CG);
    if (items == 0) return hipSuccess;
    const long long wgs = (items + T - 1) / T;
    const dim3 grid((unsigned)(wgs < (1 << 20) ? wgs : (1 << 20)));
    if (bf16)
        hipLaunchKernelGGL(k_dropout_generic<bf16_t>, grid, dim3(T), 0, s, a);
    else
        hipLaunchKernelGGL(k_dropout_generic<float>, grid, dim3(T), 0, s, a);
    return hipGetLastError();
}

}  // namespace wtc
