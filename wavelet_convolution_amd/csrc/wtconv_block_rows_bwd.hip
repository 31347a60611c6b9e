// Row kernels of the block operators, backward.
#include "wtconv_block_rows.h"

namespace wtc {
namespace {

// Over the rows of one gate (all of them, or a sample's): with e = dy where it
// is kept, S1 = sum e z and S0 = sum e give
//   dw = g k S1, db = g k S0, dg = k (w S1 + b S0)          (k: D's factor),
// so the loop adds two sums, whatever is wanted. Where every row has a gate
// of its own (HW = 1), e holds the gate and dg is written row by row.
template <typename TH, typename TY, int L, int NV, bool X, bool DROP, bool ODD>
__global__ __launch_bounds__(threads_of(L)) void k_rows_bwd(BlockArgs a, Partition pt, SumSlots sl, float* slots) {
    constexpr int T = threads_of(L), NG = T / L, W = L * NV * CG;   // W: channels that the lanes hold
    constexpr bool HOIST = NV == 1;
    __shared__ float red[L > 64 ? 4 * T / 64 : 1];
    // with a gate per sample: dw, db [2][W]; then, where NG > 1, one sum of each group [NG][W]
    extern __shared__ float lds[];
    RowSum<L> sum{red};
    const int lane = threadIdx.x % L, gi = threadIdx.x / L;
    const Lanes<L, NV, ODD> at(a.C, lane);
    const bool by_sample = X && (a.flags & BY_SAMPLE), each_row = X && (a.flags & EACH_ROW);
    float *acc = lds, *join = lds + (by_sample ? 2 * W : 0);
    // rows of a sample of the partition (all rows, unless samples count)
    const long long rows = (long long)a.B * a.HW, rps = by_sample ? a.HW : rows;
    float s1[NV][CG] = {}, s0[NV][CG] = {}, sx[NV][CG] = {};
    if (by_sample) {
        for (int e = threadIdx.x; e < 2 * W; e += T) acc[e] = 0.f;
        __syncthreads();
    }
    float* slot = slots + (size_t)blockIdx.x * (pt.nsum + pt.partials) * a.C;
    // A sum over the workgroup's rows, channel by channel. NG > 1: the groups'
    // sums meet in LDS, and channel e is then thread e % T's, in CH chains that
    // join pairwise: one chain over the 512 groups of narrow rows lost up to
    // nine bits (and took longer).
    constexpr int PER = NG > 1 ? cdiv(W, T) : 1, CH = NG < 16 ? NG : 16;
    auto joined = [&](const float (&s)[NV][CG], float (&t)[PER]) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (at.on[v])
#pragma unroll
                for (int i = 0; i < CG; ++i) join[gi * W + at.c[v] + i] = s[v][i];
        __syncthreads();
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            float p[CH] = {};
            const int e = threadIdx.x + q * T;
            if (e < a.C)
                for (int g = 0; g < NG; g += CH)
#pragma unroll
                    for (int k = 0; k < CH; ++k) p[k] += join[(g + k) * W + e];
#pragma unroll
            for (int n = CH / 2; n > 0; n /= 2)
#pragma unroll
                for (int k = 0; k < n; ++k) p[k] += p[k + n];
            t[q] = p[0];
        }
    };
    // What a gate's rows give: dg, and parts of dw and db, which add up in LDS
    // where there is a gate per sample (each place is one thread's).
    auto finish = [&](const float* gate, float* dgp) {
        if constexpr (NG > 1) {
            float t1[PER], t0[PER];
            joined(s1, t1);
            joined(s0, t0);
#pragma unroll
            for (int q = 0; q < PER; ++q) {
                const int e = threadIdx.x + q * T;
                if (e >= a.C) continue;
                if (X && dgp) {   // without a bias no 0 times S0: where dout is infinite that is no 0
                    const float w = a.w ? a.w[e] : 1.f;
                    dgp[e] = a.keep * (a.b ? w * t1[q] + a.b[e] * t0[q] : w * t1[q]);
                }
                const float g = X ? (gate ? gate[e] : 1.f) * a.keep : 1.f;
                if (by_sample) {
                    acc[e] += g * t1[q];
                    acc[W + e] += g * t0[q];
                } else {
                    if (sl.dw >= 0) slot[(size_t)sl.dw * a.C + e] = g * t1[q];
                    if (sl.db >= 0) slot[(size_t)sl.db * a.C + e] = g * t0[q];
                }
            }
        } else {   // channels that two lanes share are the same in both
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (!at.on[v]) continue;
                float p[CG], q[CG];
                if (X && dgp) {
                    at.param(a.w, v, 1.f, p);
                    at.param(a.b, v, 0.f, q);
#pragma unroll
                    for (int i = 0; i < CG; ++i)
                        p[i] = a.keep * (a.b ? p[i] * s1[v][i] + q[i] * s0[v][i] : p[i] * s1[v][i]);
                    at.store(dgp, p, v);
                }
                float g[CG];
                at.param(gate, v, 1.f, g);
                float* mine = acc + (v * L + lane) * CG;
#pragma unroll
                for (int i = 0; i < CG; ++i) {
                    if constexpr (X) g[i] *= a.keep;
                    p[i] = g[i] * s1[v][i];
                    q[i] = g[i] * s0[v][i];
                    if (by_sample) {
                        mine[i] += p[i];
                        mine[W + i] += q[i];
                    }
                }
                if (!by_sample && sl.dw >= 0) at.store(slot + (size_t)sl.dw * a.C, p, v);
                if (!by_sample && sl.db >= 0) at.store(slot + (size_t)sl.db * a.C, q, v);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    // u = e gw; kept in registers while it does not change
    float gw[NV][CG];
    auto gates = [&](int v, const float* gate) {
        at.param(a.w, v, 1.f, gw[v]);
        if constexpr (X) {
            float g[CG];
            at.param(gate, v, 1.f, g);
#pragma unroll
            for (int i = 0; i < CG; ++i) gw[v][i] *= g[i] * a.keep;
        }
    };
    const long long t0 = pt.begin(blockIdx.x), t1 = pt.begin(blockIdx.x + 1);
    long long s = by_sample ? t0 / pt.tps : 0, j = t0 - s * pt.tps;   // sample, tile in it
    bool fresh = true;   // another gate than the last tile's
    for (long long t = t0; t < t1; ++t) {
        uint32_t fl = a.flags;
        asm volatile("" : "+s"(fl));   // tested here, not before the loop
        const long long r0 = j * NG + gi, row = s * rps + r0;
        const bool live = r0 < rps;
        const int bi = !X || !live ? 0 : by_sample ? (int)s : fl & DROPS_SAMPLES ? sample_of(a, row) : 0;
        const bool in = live && (!X || !(fl & DROPS_SAMPLES) || sample_kept(a, bi));
        Vec<TH, CG> hv[NV];
        Vec<TY, CG> dv[NV], x[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            hv[v].zero();
            if (in && at.on[v]) at.load(hv[v], (const TH*)a.h + row * a.C, v);
            dv[v].zero();
            if (live && at.on[v]) at.load(dv[v], (const TY*)a.dy + row * a.C, v);
            if (X && (fl & WANT_DXS) && live && at.on[v]) at.load(x[v], (const TY*)a.x + row * a.C, v);
        }
        if (!each_row && fresh) {
            fresh = false;
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (HOIST && at.on[v]) gates(v, by_sample ? a.gate + s * a.C : a.gate);
        }
        float h[NV][CG], d[NV][CG];
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < CG; ++i) {
                h[v][i] = hv[v][i];
                d[v][i] = dv[v][i];
            }
        if constexpr (X) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (!live || !at.on[v]) continue;
                if (fl & WANT_DXS) {
#pragma unroll
                    for (int i = 0; i < CG; ++i) sx[v][i] = fmaf(d[v][i], x[v][i], sx[v][i]);
                }
                if (fl & WANT_DX) {
                    float xs[CG], o[CG];
                    at.param(a.xs, v, 1.f, xs);
#pragma unroll
                    for (int i = 0; i < CG; ++i) o[i] = d[v][i] * xs[i];
                    at.store((TY*)a.dx + row * a.C, o, v);
                }
            }
        }
        float mean = 0.f, r = 1.f;
        if (fl & (LAYER | RMS)) row_stats<L, NV, ODD>(a, fl & LAYER, h, at, sum, mean, r);
        float m1 = 0.f, m2 = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (!live || !at.on[v]) continue;
            if (X && !in) {   // no gradient passes a dropped sample
#pragma unroll
                for (int i = 0; i < CG; ++i) d[v][i] = 0.f;
            }
            if constexpr (DROP) {
                const uint32_t m = drop_bits_at(Philox(a.rng, a.site), (uint32_t)row * (uint32_t)cdiv(a.C, CG),
                                                at.c[v], ODD, a.thr);
#pragma unroll
                for (int i = 0; i < CG; ++i) d[v][i] = kept(d[v][i], m, i);
                if (!(fl & (LAYER | RMS))) {   // 0 times NaN is no 0
#pragma unroll
                    for (int i = 0; i < CG; ++i) h[v][i] = kept(h[v][i], m, i);
                }
            }
#pragma unroll
            for (int i = 0; i < CG; ++i) h[v][i] = (h[v][i] - mean) * r;   // z from here on
            if (X && each_row) {
                float w[CG], b[CG], g[CG], o[CG];
                at.param(a.w, v, 1.f, w);
                at.param(a.b, v, 0.f, b);
                at.param(a.gate + row * a.C, v, 1.f, g);
#pragma unroll
                for (int i = 0; i < CG; ++i) {
                    o[i] = d[v][i] * fmaf(h[v][i], w[i], b[i]) * a.keep;
                    gw[v][i] = w[i] * a.keep;
                    d[v][i] *= g[i];
                }
                if (a.dg) at.store(a.dg + row * a.C, o, v);
            } else if constexpr (!HOIST) {
                gates(v, by_sample ? a.gate + s * a.C : a.gate);
            }
#pragma unroll
            for (int i = 0; i < CG; ++i) {
                s1[v][i] = fmaf(d[v][i], h[v][i], s1[v][i]);
                s0[v][i] += d[v][i];
                d[v][i] *= gw[v][i];   // u from here on
                const float u = at.once(d[v][i], v, i);
                m1 += u;
                m2 = fmaf(u, h[v][i], m2);
                asm volatile("" : "+v"(s1[v][i]), "+v"(s0[v][i]));   // here, not where they are used
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (fl & WANT_DH) {
            if (fl & (LAYER | RMS)) {
                sum.two(m1, m2);
                m1 = fl & LAYER ? m1 * a.inv_c : 0.f;
                m2 *= a.inv_c;
            }
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (!live || !at.on[v]) continue;
                float o[CG];
#pragma unroll
                for (int i = 0; i < CG; ++i) o[i] = fl & (LAYER | RMS) ? r * (d[v][i] - m1 - h[v][i] * m2) : d[v][i];
                at.store((TH*)a.dh + row * a.C, o, v);
            }
        }
        if (++j == pt.tps && by_sample) {
            j = 0;
            fresh = true;
        }
        // the last tile of this sample in the workgroup's range
        if (by_sample && (t + 1 == t1 || j == 0)) {
            const bool whole = s * pt.tps >= t0 && (s + 1) * pt.tps <= t1;
            finish(a.gate + s * a.C,
                   !a.dg   ? nullptr
                   : whole ? a.dg + s * a.C
                           : slot + (size_t)(pt.nsum + (s == t0 / pt.tps ? 0 : 1)) * a.C);
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < CG; ++i) s1[v][i] = s0[v][i] = 0.f;
            if (j == 0) ++s;
        }
    }
    if (!by_sample) {
        finish(each_row ? nullptr : a.gate, sl.dg >= 0 ? slot + (size_t)sl.dg * a.C : nullptr);
    } else if constexpr (NG > 1) {
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int e = threadIdx.x + q * T;
            if (e >= a.C) continue;
            if (sl.dw >= 0) slot[(size_t)sl.dw * a.C + e] = acc[e];
            if (sl.db >= 0) slot[(size_t)sl.db * a.C + e] = acc[W + e];
        }
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (!at.on[v]) continue;
            float p[CG], q[CG];
#pragma unroll
            for (int i = 0; i < CG; ++i) {
                p[i] = acc[(v * L + lane) * CG + i];
                q[i] = acc[W + (v * L + lane) * CG + i];
            }
            if (sl.dw >= 0) at.store(slot + (size_t)sl.dw * a.C, p, v);
            if (sl.db >= 0) at.store(slot + (size_t)sl.db * a.C, q, v);
        }
    }
    if (X && sl.dxs >= 0) {
        float* to = slot + (size_t)sl.dxs * a.C;
        if constexpr (NG > 1) {
            float tx[PER];
            joined(sx, tx);
#pragma unroll
            for (int q = 0; q < PER; ++q)
                if ((int)threadIdx.x + q * T < a.C) to[threadIdx.x + q * T] = tx[q];
        } else {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (at.on[v]) at.store(to, sx[v], v);
        }
    }
}

template <int L, int NV>
struct Groups {
    static Partition call(const BlockArgs* a) {
        constexpr int T = threads_of(L), NG = T / L;
        Partition p{};
        // a tile: the rows that a workgroup takes at once
        const bool by_sample = a->gate_mode == GATE_SAMPLE && a->HW > 1;
        const long long rows = (long long)a->B * a->HW, rps = by_sample ? a->HW : rows;
        p.tps = (rps + NG - 1) / NG;
        p.tiles = by_sample ? a->B * p.tps : p.tps;
        // as many workgroups as the card holds at once, sixteen wavefronts a CU
        // (more write more partial sums: 8,192 x 4,096 bf16 with an fp32 stream,
        // 70 us at 512 workgroups, 84 at 768, 102 at 2,048)
        const long long wgs = 256 * (1024 / T);
        p.wgs = (int)(p.tiles < wgs ? p.tiles : wgs);
        p.nsum = sum_slots(*a).count;
        p.partials = by_sample && a->dg && p.tps > 1 ? 2 : 0;
        return p;
    }
};
Partition rows_partition(const BlockArgs& a) {
    return block_residual(a) ? for_row<Groups, true>(a.C, &a) : for_row<Groups, false>(a.C, &a);
}

template <typename TH, typename TY, bool X, bool DROP, bool ODD>
struct Bwd {
    template <int L, int NV>
    struct F {
        static hipError_t call(const BlockArgs* a, const Partition* p, hipStream_t s) {
            constexpr int T = threads_of(L), W = L * NV * CG;
            const size_t lds = sizeof(float) * ((a->flags & BY_SAMPLE ? 2 * W : 0) + (T / L > 1 ? T / L * W : 0));
            hipLaunchKernelGGL((k_rows_bwd<TH, TY, L, NV, X, DROP, ODD>), dim3((unsigned)p->wgs), dim3(T), lds, s, *a,
                               *p, sum_slots(*a), a->ws);
            return hipGetLastError();
        }
    };
};

}  // namespace

// (With every gradient wanted, which a size is asked for, a call counts as a
// residual's: its tiles are the smaller ones and its workgroups the more.)
size_t rows_bwd_bytes(const BlockArgs& a) {
    const Partition p = rows_partition(a);
    return (size_t)p.wgs * (p.nsum + p.partials) * a.C * sizeof(float);
}

hipError_t rows_bwd(const BlockArgs& args, int h_bf16, int y_bf16, hipStream_t s) {
    BlockArgs a = args;
    a.flags = block_flags(a);
    const Partition p = rows_partition(a);
    if (p.wgs > 0) {
        const hipError_t err = by_type<Bwd, true>(a, h_bf16, y_bf16, block_residual(a), &p, s);
        if (err != hipSuccess) return err;
    }
    return block_finalize(a, p, a.ws, s);
}

}  // namespace wtc
