// Counter dropout: y = keep ? x * 65536 / (65536 - thr) : 0, the mask computed
// from (seed, offset, site, element) and never stored; the backward pass is
// the same call on dy. A generator call serves the eight channels of a group
// and runs while the loads are in flight: 20 quarter-rate products and about
// 80 other instructions for eight elements are 0.4 us a million elements
// (bf16: 0.77 us at the copy rate), so memory is the bound.
#include "wtconv_block_device.h"

namespace wtc {
namespace {

constexpr int T = 256;

// Rows (channels last): a thread takes groups of eight channels, G to a row,
// each one vector; where C is no multiple of eight (ODD), the last one of a
// row moves back to end with it, over two of the generator's groups.
constexpr int UNROLL = 2;
template <typename X, bool ODD>
__global__ __launch_bounds__(T) void k_dropout_rows(BlockArgs a, uint32_t items, uint32_t G) {
    const X* h = (const X*)a.h;
    X* y = (X*)a.y;
    const Philox gen(a.rng, a.site);
    const uint32_t step = gridDim.x * T;   // below 2^31
    for (uint32_t n = blockIdx.x * T + threadIdx.x; n < items;) {
        Vec<X, CG> v[UNROLL];
        size_t at[UNROLL];
        uint32_t m[UNROLL];
        uint32_t k[UNROLL];
        bool on[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            k[u] = n;
            on[u] = u == 0 || n < items;
            if (on[u]) {
                if constexpr (ODD) {
                    const uint32_t row = n / G, c = min((n - row * G) * CG, (uint32_t)a.C - CG);
                    at[u] = (size_t)row * a.C + c;
                } else {
                    at[u] = (size_t)n * CG;
                }
                v[u].load(h + at[u]);
            }
            n = on[u] && items - n > step ? n + step : items;   // no sum past 2^32
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            if constexpr (ODD) {
                const uint32_t row = k[u] / G;
                m[u] = drop_bits_at(gen, row * G, (int)(at[u] - (size_t)row * a.C), true, a.thr);
            } else {
                m[u] = drop_bits(gen(k[u]), a.thr);
            }
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            if (!on[u]) continue;
            float o[CG];
#pragma unroll
            for (int i = 0; i < CG; ++i) o[i] = kept(v[u][i] * a.keep, m[u], i);
            store_vec<X, CG>(y + at[u], o);
        }
    }
}

// Planes: a thread takes PV consecutive pixels of a group's eight channels, a
// generator call for each pixel; the last pixels of a plane and the last
// channels of a sample move back to end with them.
template <typename X, int PV, bool ODD>
__global__ __launch_bounds__(T) void k_dropout_planes(BlockArgs a, uint32_t items, uint32_t G, uint32_t vecs) {
    for (uint64_t n64 = (uint64_t)blockIdx.x * T + threadIdx.x; n64 < items; n64 += (uint64_t)gridDim.x * T) {
        const uint32_t n = (uint32_t)n64, bg = n / vecs, p = min((n - bg * vecs) * PV, (uint32_t)a.HW - PV);
        const uint32_t b = bg / G, c = min((bg - b * G) * CG, (uint32_t)a.C - CG);
        const size_t at = ((size_t)b * a.C + c) * a.HW + p;
        Patch<X, false, PV> v;
        v.load((const X*)a.h + at, 0, a.HW);
        Drops<PV> drop;
        drop.template draw<ODD>(a, b * a.HW + p, (int)c);
        v.drop(drop);
        store_patch<X, false, PV>((X*)a.y + at, 0, a.HW, [&](int i, int j) { return v.at(i, j) * a.keep; });
    }
}

// Whole samples: contiguous in either order, `vecs` vectors each (the last one
// moved back); a dropped sample's x is not read.
template <typename X>
__global__ __launch_bounds__(T) void k_dropout_samples(BlockArgs a, uint64_t size, uint32_t vecs) {
    const uint64_t items = (uint64_t)a.B * vecs;
    for (uint64_t n = (uint64_t)blockIdx.x * T + threadIdx.x; n < items; n += (uint64_t)gridDim.x * T) {
        const uint32_t b = (uint32_t)(n / vecs);
        const uint64_t e = (uint64_t)(n - (uint64_t)b * vecs) * CG;
        const size_t at = b * size + (e < size - CG ? e : size - CG);
        Vec<X, CG> v;
        v.zero();
        if (sample_kept(a, (int)b)) v.load((const X*)a.h + at);
        float o[CG];
#pragma unroll
        for (int i = 0; i < CG; ++i) o[i] = v[i] * a.keep;
        store_vec<X, CG>((X*)a.y + at, o);
    }
}

// Any size: a thread takes the channels of one group in one row, one by one.
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

unsigned grid_of(uint64_t items, uint64_t most) {
    const uint64_t wgs = (items + T - 1) / T;
    return (unsigned)(wgs < most ? wgs : most);
}

template <typename X, int PV>
hipError_t launch(const BlockArgs& a, hipStream_t s) {
    const uint64_t G = cdiv(a.C, CG), rows = (uint64_t)a.B * a.HW, size = (uint64_t)a.C * a.HW;
    if (rows == 0) return hipSuccess;
    if (a.drop == DROP_SAMPLE && size >= CG && size <= (uint64_t)0xffffffffu) {
        const uint32_t vecs = (uint32_t)((size + CG - 1) / CG);
        hipLaunchKernelGGL(k_dropout_samples<X>, dim3(grid_of((uint64_t)a.B * vecs, 1 << 20)), dim3(T), 0, s, a, size,
                           vecs);
    } else if (a.drop == DROP_ELEMENT && a.h_cl && a.C >= CG) {
        // eight workgroups a CU, each thread with several groups
        const dim3 grid(grid_of((rows * G + UNROLL - 1) / UNROLL, 256 * 8));
        if (a.C % CG)
            hipLaunchKernelGGL((k_dropout_rows<X, true>), grid, dim3(T), 0, s, a, (uint32_t)(rows * G), (uint32_t)G);
        else
            hipLaunchKernelGGL((k_dropout_rows<X, false>), grid, dim3(T), 0, s, a, (uint32_t)(rows * G), (uint32_t)G);
    } else if (a.drop == DROP_ELEMENT && !a.h_cl && a.C >= CG && a.HW >= PV) {
        const uint32_t vecs = (uint32_t)cdiv(a.HW, PV);
        const uint64_t items = (uint64_t)a.B * G * vecs;   // fewer than the groups: below 2^32
        const dim3 grid(grid_of(items, 1 << 20));
        if (a.C % CG)
            hipLaunchKernelGGL((k_dropout_planes<X, PV, true>), grid, dim3(T), 0, s, a, (uint32_t)items, (uint32_t)G,
                               vecs);
        else
            hipLaunchKernelGGL((k_dropout_planes<X, PV, false>), grid, dim3(T), 0, s, a, (uint32_t)items, (uint32_t)G,
                               vecs);
    } else {
        hipLaunchKernelGGL(k_dropout_generic<X>, dim3(grid_of(rows * G, 1 << 20)), dim3(T), 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t dropout_launch(const BlockArgs& a, int bf16, hipStream_t s) {
    return bf16 ? launch<bf16_t, 8>(a, s) : launch<float, 4>(a, s);
}

}  // namespace wtc
