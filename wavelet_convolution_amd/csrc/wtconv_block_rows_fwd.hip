// Row kernels of the block operators, forward.
#include "wtconv_block_rows.h"

namespace wtc {
namespace {

// X: a residual (else a norm alone); DROP: elements are dropped.
template <typename TH, typename TY, int L, int NV, bool X, bool DROP, bool ODD>
__global__ __launch_bounds__(threads_of(L)) void k_rows_fwd(BlockArgs a) {
    constexpr int T = threads_of(L), NG = T / L;
    constexpr bool HOIST = NV == 1;   // parameters in registers over the rows
    __shared__ float red[L > 64 ? 4 * T / 64 : 1];
    RowSum<L> sum{red};
    const Lanes<L, NV, ODD> at(a.C, threadIdx.x % L);
    const int gi = threadIdx.x / L;
    const long long rows = (long long)a.B * a.HW;
    // y = s x + D'(z wg + bg), with the gate and D's factor in wg and bg
    float wg[CG], bg[CG], xs[CG];
    const bool by_sample = X && a.gate_mode == GATE_SAMPLE;
    auto params = [&](int v, long long bi) {
        at.param(a.w, v, 1.f, wg);
        at.param(a.b, v, 0.f, bg);
        if constexpr (X) {
            float g[CG];
            at.param(a.xs, v, 1.f, xs);
            at.param(by_sample ? a.gate + bi * a.C : a.gate, v, 1.f, g);
#pragma unroll
            for (int i = 0; i < CG; ++i) {
                g[i] *= a.keep;
                wg[i] *= g[i];
                bg[i] *= g[i];
            }
        }
    };
    if (HOIST && !by_sample && at.on[0]) params(0, 0);
    for (long long r0 = (long long)blockIdx.x * NG; r0 < rows; r0 += (long long)gridDim.x * NG) {
        const long long row = r0 + gi;
        const bool live = row < rows;
        const int bi = X && live && (by_sample || a.drop == DROP_SAMPLE) ? sample_of(a, row) : 0;
        const bool in = live && (!X || a.drop != DROP_SAMPLE || sample_kept(a, bi));
        Vec<TH, CG> hv[NV];
        Vec<TY, CG> x[NV];
        float h[NV][CG];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            hv[v].zero();   // a dropped sample's h is not looked at
            if (in && at.on[v]) at.load(hv[v], (const TH*)a.h + row * a.C, v);
            if (X && live && at.on[v]) at.load(x[v], (const TY*)a.x + row * a.C, v);
        }
        if (HOIST && by_sample && at.on[0]) params(0, bi);
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < CG; ++i) h[v][i] = hv[v][i];
        float mean = 0.f, r = 1.f;
        if (a.norm != NORM_NONE) row_stats<L, NV, ODD>(a, a.norm == NORM_LAYER, h, at, sum, mean, r);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (!live || !at.on[v]) continue;
            if constexpr (!HOIST) params(v, bi);
            float o[CG];
#pragma unroll
            for (int i = 0; i < CG; ++i) o[i] = fmaf((h[v][i] - mean) * r, wg[i], bg[i]);
            if constexpr (DROP) {
                const uint32_t m = drop_bits_at(Philox(a.rng, a.site), (uint32_t)row * (uint32_t)cdiv(a.C, CG),
                                                at.c[v], ODD, a.thr);
#pragma unroll
                for (int i = 0; i < CG; ++i) o[i] = kept(o[i], m, i);
            }
            if constexpr (X) {
#pragma unroll
                for (int i = 0; i < CG; ++i) o[i] = fmaf(xs[i], x[v][i], in ? o[i] : 0.f);
            }
            at.store((TY*)a.y + row * a.C, o, v);
        }
    }
}

template <typename TH, typename TY, bool X, bool DROP, bool ODD>
struct Fwd {
    template <int L, int NV>
    struct F {
        static hipError_t call(const BlockArgs* a, hipStream_t s) {
            constexpr int T = threads_of(L), NG = T / L;
            const long long rows = (long long)a->B * a->HW, wgs = (rows + NG - 1) / NG, most = 256 * (2048 / T);
            hipLaunchKernelGGL((k_rows_fwd<TH, TY, L, NV, X, DROP, ODD>), dim3((unsigned)(wgs < most ? wgs : most)),
                               dim3(T), 0, s, *a);
            return hipGetLastError();
        }
    };
};

}  // namespace

bool rows_cover(const BlockArgs& a) { return a.h_cl && a.y_cl && a.C <= 2048 * CG; }

hipError_t rows_fwd(const BlockArgs& a, int h_bf16, int y_bf16, hipStream_t s) {
    if ((long long)a.B * a.HW == 0) return hipSuccess;
    return by_type<Fwd, false>(a, h_bf16, y_bf16, a.x != nullptr, s);
}

}  // namespace wtc
