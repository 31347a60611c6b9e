// Block operators on rows: both sides channels last (or tokens). A row of C
// channels is held in the registers of L lanes, NV vectors of eight channels
// a lane, from its one read to its store; the mean, the variance about it and
// the two means of the backward pass are sums over those lanes (within a
// wavefront by data-parallel moves, L > 64 through LDS). A workgroup takes
// several rows at once where L is small, and loops over its rows, so a lane's
// channels never change: parameters are loaded once (NV = 1), and parameter
// gradients add up in registers, then over the workgroup's rows in LDS, then
// over workgroups in the second stage.
// Bound by memory: 2 + 2 (+ 2) bytes an element forwards in bf16.
#include "wtconv_block_device.h"

namespace wtc {
namespace {

constexpr int threads_of(int L) { return L < 256 ? 256 : L; }

// Sum over a row's L lanes. L > 64: the wavefronts' sums meet in LDS, in one
// of two buffers in turn (one barrier a sum: a buffer is written again only
// after the barrier of the sum in between).
template <int L>
struct RowSum {
    float* red;   // [2][2][L / 64]
    int turn = 0;
    __device__ __forceinline__ float one(float v) {
        if constexpr (L <= 64) {
            return lane_sum<L>(v);
        } else {
            constexpr int W = L / 64;
            float* buf = red + turn * 2 * W;
            turn ^= 1;
            v = lane_sum<64>(v);
            if (threadIdx.x % 64 == 0) buf[threadIdx.x / 64] = v;
            __syncthreads();
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) s += buf[i];
            return s;
        }
    }
    __device__ __forceinline__ void two(float& a, float& b) {
        if constexpr (L <= 64) {
            a = lane_sum<L>(a);
            b = lane_sum<L>(b);
        } else {
            constexpr int W = L / 64;
            float* buf = red + turn * 2 * W;
            turn ^= 1;
            a = lane_sum<64>(a);
            b = lane_sum<64>(b);
            if (threadIdx.x % 64 == 0) {
                buf[threadIdx.x / 64] = a;
                buf[W + threadIdx.x / 64] = b;
            }
            __syncthreads();
            a = b = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                a += buf[i];
                b += buf[W + i];
            }
        }
    }
};

// mean and r of a row: the variance about the mean in a second sum over the
// registers (no difference of large sums). Channels past C do not count.
template <typename TH, int NV, int L>
__device__ __forceinline__ void row_stats(const BlockArgs& a, const Vec<TH, CG> (&h)[NV], const int (&n)[NV],
                                          RowSum<L>& sum, float& mean, float& r) {
    mean = 0.f;
    r = 1.f;
    if (a.norm == NORM_NONE) return;
    const float inv = 1.f / (float)a.C;
    if (a.norm == NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < CG; ++i) s += h[v][i];   // zeros past C
        mean = sum.one(s) * inv;
    }
    float q = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < CG; ++i) {
            const float d = i < n[v] ? h[v][i] - mean : 0.f;
            q = fmaf(d, d, q);
        }
    r = 1.f / sqrtf(sum.one(q) * inv + a.eps);
}

template <typename TH, typename TY, int L, int NV>
__global__ __launch_bounds__(threads_of(L)) void k_rows_fwd(BlockArgs a) {
    constexpr int T = threads_of(L), NG = T / L;
    constexpr bool HOIST = NV == 1;
    __shared__ float red[L > 64 ? 4 * L / 64 : 1];
    RowSum<L> sum{red};
    const int lane = threadIdx.x % L, gi = threadIdx.x / L;
    const long long rows = (long long)a.B * a.HW;
    const uint32_t G = (uint32_t)cdiv(a.C, CG);
    int c[NV], n[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        c[v] = (v * L + lane) * CG;
        n[v] = max(0, min(CG, a.C - c[v]));
    }
    float w[CG], b[CG], gt[CG], xs[CG];
    const bool by_sample = a.gate_mode == GATE_SAMPLE;
    auto params = [&](int v, long long bi) {
        load_param(a.w, c[v], n[v], 1.f, w);
        load_param(a.b, c[v], n[v], 0.f, b);
        load_param(a.xs, c[v], n[v], 1.f, xs);
        load_param(by_sample ? a.gate + bi * a.C : a.gate, c[v], n[v], 1.f, gt);
    };
    if constexpr (HOIST) {
        if (a.w) load_param(a.w, c[0], n[0], 1.f, w);
        if (a.b) load_param(a.b, c[0], n[0], 0.f, b);
        if (a.xs) load_param(a.xs, c[0], n[0], 1.f, xs);
        if (a.gate && !by_sample) load_param(a.gate, c[0], n[0], 1.f, gt);
    }
    for (long long r0 = (long long)blockIdx.x * NG; r0 < rows; r0 += (long long)gridDim.x * NG) {
        const long long row = r0 + gi;
        const bool live = row < rows;
        const long long bi = by_sample || a.drop == DROP_SAMPLE ? (live ? row / a.HW : 0) : 0;
        const bool kept = live && (a.drop != DROP_SAMPLE || sample_kept(a, (int)bi));
        const TH* hp = (const TH*)a.h + row * a.C;
        const TY* xp = (const TY*)a.x + row * a.C;
        Vec<TH, CG> h[NV];
        Vec<TY, CG> x[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            h[v].zero();   // a dropped sample's h is not looked at
            if (kept && n[v] > 0) h[v].load(hp + c[v], n[v]);
            x[v].zero();
            if (a.x && live && n[v] > 0) x[v].load(xp + c[v], n[v]);
        }
        if constexpr (HOIST)
            if (by_sample && live && n[0] > 0) load_param(a.gate + bi * a.C, c[0], n[0], 1.f, gt);
        float mean, r;
        row_stats<TH, NV, L>(a, h, n, sum, mean, r);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (!live || n[v] <= 0) continue;
            if constexpr (!HOIST) params(v, bi);
            uint32_t m = kept ? 0xffu : 0u;
            if (a.drop == DROP_ELEMENT) {
                const Philox gen(a.rng, a.site);
                m = keep_bits(gen((uint32_t)row * G + (uint32_t)(c[v] / CG)), a.thr);
            }
            float o[CG];
#pragma unroll
            for (int i = 0; i < CG; ++i) {
                o[i] = (h[v][i] - mean) * r;
                if (!HOIST || a.w) o[i] *= w[i];
                if (!HOIST || a.b) o[i] += b[i];
                if (a.drop != DROP_NONE) o[i] = m >> i & 1 ? o[i] * a.keep : 0.f;
                if (!HOIST || a.gate) o[i] *= gt[i];
                if (a.x) o[i] += !HOIST || a.xs ? xs[i] * x[v][i] : x[v][i];
            }
            store_vec<TY, CG>((TY*)a.y + row * a.C + c[v], o, n[v]);
        }
    }
}

template <typename TH, typename TY, int L, int NV>
__global__ __launch_bounds__(threads_of(L)) void k_rows_bwd(BlockArgs a, Partition pt, SumSlots sl, float* slots) {
    constexpr int T = threads_of(L), NG = T / L;
    __shared__ float red[L > 64 ? 4 * L / 64 : 1];
    __shared__ float join[NG > 1 ? NG * L * NV * CG : 1];
    RowSum<L> sum{red};
    const int lane = threadIdx.x % L, gi = threadIdx.x / L;
    const uint32_t G = (uint32_t)cdiv(a.C, CG);
    const bool sample_gate = a.gate_mode == GATE_SAMPLE;
    const bool each_row = a.dg && sample_gate && a.HW == 1;   // a row is a sample: its gate gradient is written at once
    const bool by_sample = a.dg && sample_gate && !each_row;
    // rows of a sample of the partition (all rows, unless samples count)
    const long long rows = (long long)a.B * a.HW, rps = by_sample ? a.HW : rows;
    int c[NV], n[NV];
    float dw[NV][CG] = {}, db[NV][CG] = {}, dg[NV][CG] = {}, ds[NV][CG] = {};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        c[v] = (v * L + lane) * CG;
        n[v] = max(0, min(CG, a.C - c[v]));
    }
    float* slot = slots + (size_t)blockIdx.x * (pt.nsum + pt.partials) * a.C;
    // sums over the workgroup's groups of lanes, in order, then out
    auto put = [&](float (&s)[NV][CG], float* to) {
        if constexpr (NG > 1) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < CG; ++i) join[(gi * NV + v) * L * CG + lane * CG + i] = s[v][i];
            __syncthreads();
            for (int e = threadIdx.x; e < NV * L * CG; e += T) {
                float t = 0.f;
#pragma unroll
                for (int g = 0; g < NG; ++g) t += join[g * NV * L * CG + e];
                if (e < a.C) to[e] = t;   // element e of the lanes' vectors is channel e
            }
        } else {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (n[v] > 0) store_vec<float, CG>(to + c[v], s[v], n[v]);
        }
    };
    const long long t0 = blockIdx.x * pt.per_wg, t1 = min(t0 + pt.per_wg, pt.tiles);
    for (long long t = t0; t < t1; ++t) {
        const long long s = by_sample ? t / pt.tps : 0, in = (t - s * pt.tps) * NG + gi, row = s * rps + in;
        const bool live = in < rps;
        const long long bi = by_sample ? s : sample_gate || a.drop == DROP_SAMPLE ? (live ? row / a.HW : 0) : 0;
        const bool kept = live && (a.drop != DROP_SAMPLE || sample_kept(a, (int)bi));
        Vec<TH, CG> h[NV];
        Vec<TY, CG> d[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            h[v].zero();
            if (kept && n[v] > 0) h[v].load((const TH*)a.h + row * a.C + c[v], n[v]);
            d[v].zero();
            if (live && n[v] > 0) d[v].load((const TY*)a.dy + row * a.C + c[v], n[v]);
        }
        float mean, r;
        row_stats<TH, NV, L>(a, h, n, sum, mean, r);
        float m1 = 0.f, m2 = 0.f;
        float dv[NV][CG];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float w[CG], b[CG], gt[CG];
            const bool on = live && n[v] > 0;
            load_param(on ? a.w : nullptr, c[v], n[v], 1.f, w);
            load_param(on ? a.b : nullptr, c[v], n[v], 0.f, b);
            load_param(!on ? nullptr : sample_gate ? a.gate + bi * a.C : a.gate, c[v], n[v], 1.f, gt);
            uint32_t m = kept ? 0xffu : 0u;
            if (a.drop == DROP_ELEMENT && on) {
                const Philox gen(a.rng, a.site);
                m = keep_bits(gen((uint32_t)row * G + (uint32_t)(c[v] / CG)), a.thr);
            }
            float row_dg[CG];
#pragma unroll
            for (int i = 0; i < CG; ++i) {
                const bool k = m >> i & 1;
                const float z = (h[v][i] - mean) * r, di = d[v][i];   // di = 0 past C
                dv[v][i] = k ? di * gt[i] * a.keep : 0.f;
                row_dg[i] = k ? di * (fmaf(z, w[i], b[i]) * a.keep) : 0.f;
                dw[v][i] = fmaf(dv[v][i], z, dw[v][i]);
                db[v][i] += dv[v][i];
                dg[v][i] += row_dg[i];
                dv[v][i] *= w[i];   // u from here on
                m1 += dv[v][i];
                m2 = fmaf(dv[v][i], z, m2);
            }
            if (each_row && on) store_vec<float, CG>(a.dg + row * a.C + c[v], row_dg, n[v]);
        }
        if (a.norm != NORM_NONE && a.dh) {
            const float inv = 1.f / (float)a.C;
            sum.two(m1, m2);
            m1 = a.norm == NORM_LAYER ? m1 * inv : 0.f;
            m2 *= inv;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (!live || n[v] <= 0) continue;
            if (a.dh) {
                float o[CG];
#pragma unroll
                for (int i = 0; i < CG; ++i) {
                    const float z = (h[v][i] - mean) * r;
                    o[i] = a.norm == NORM_NONE ? dv[v][i] : r * (dv[v][i] - m1 - z * m2);
                }
                store_vec<TH, CG>((TH*)a.dh + row * a.C + c[v], o, n[v]);
            }
            if (a.dx) {
                float xs[CG], o[CG];
                load_param(a.xs, c[v], n[v], 1.f, xs);
#pragma unroll
                for (int i = 0; i < CG; ++i) o[i] = d[v][i] * xs[i];
                store_vec<TY, CG>((TY*)a.dx + row * a.C + c[v], o, n[v]);
            }
            if (a.dxs) {
                Vec<TY, CG> x;
                x.load((const TY*)a.x + row * a.C + c[v], n[v]);
#pragma unroll
                for (int i = 0; i < CG; ++i) ds[v][i] = fmaf(d[v][i], x[i], ds[v][i]);
            }
        }
        // the last tile of this sample in the workgroup's range
        if (by_sample && (t + 1 == t1 || (t + 1) % pt.tps == 0)) {
            const bool whole = s * pt.tps >= t0 && (s + 1) * pt.tps <= t1;
            put(dg, whole ? a.dg + s * a.C : slot + (size_t)(pt.nsum + (s == t0 / pt.tps ? 0 : 1)) * a.C);
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < CG; ++i) dg[v][i] = 0.f;
        }
    }
    if (sl.dw >= 0) put(dw, slot + (size_t)sl.dw * a.C);
    if (sl.db >= 0) put(db, slot + (size_t)sl.db * a.C);
    if (sl.dg >= 0) put(dg, slot + (size_t)sl.dg * a.C);
    if (sl.dxs >= 0) put(ds, slot + (size_t)sl.dxs * a.C);
}

// The layouts of a row over lanes, by its vectors of eight channels: the
// fewest lanes that hold it at one vector each, then two vectors (C = 513 to
// 1024 stays within a wavefront, without a barrier), then whole workgroups.
template <template <int, int> class F, class... A>
auto for_row(int C, A... args) {
    const int vecs = cdiv(C, CG);
    if (vecs <= 1) return F<1, 1>::call(args...);
    if (vecs <= 4) return F<4, 1>::call(args...);
    if (vecs <= 8) return F<8, 1>::call(args...);
    if (vecs <= 16) return F<16, 1>::call(args...);
    if (vecs <= 32) return F<32, 1>::call(args...);
    if (vecs <= 64) return F<64, 1>::call(args...);
    if (vecs <= 128) return F<64, 2>::call(args...);
    if (vecs <= 256) return F<256, 1>::call(args...);
    if (vecs <= 512) return F<256, 2>::call(args...);
    if (vecs <= 1024) return F<512, 2>::call(args...);
    return F<1024, 2>::call(args...);
}

template <int L, int NV>
struct GroupsOf {
    static int call() { return threads_of(L) / L; }
};

// Rows at once in a workgroup; the partition's tiles are that many rows.
Partition rows_partition(const BlockArgs& a) {
    const int NG = for_row<GroupsOf>(a.C);
    Partition p{};
    const bool by_sample = a.dg && a.gate_mode == GATE_SAMPLE && a.HW > 1;
    const long long rows = (long long)a.B * a.HW, rps = by_sample ? a.HW : rows;
    p.tps = (rps + NG - 1) / NG;
    p.tiles = by_sample ? a.B * p.tps : p.tps;
    p.per_wg = (p.tiles + 1023) / 1024;
    if (p.per_wg < 4) p.per_wg = 4;
    p.wgs = (int)((p.tiles + p.per_wg - 1) / p.per_wg);
    p.nsum = sum_slots(a).count;
    p.partials = by_sample && p.per_wg % p.tps ? 2 : 0;
    return p;
}

template <typename TH, typename TY>
struct Fwd {
    template <int L, int NV>
    struct F {
        static hipError_t call(const BlockArgs* a, hipStream_t s) {
            constexpr int T = threads_of(L), NG = T / L;
            const long long rows = (long long)a->B * a->HW, wgs = (rows + NG - 1) / NG, most = 256 * (2048 / T);
            hipLaunchKernelGGL((k_rows_fwd<TH, TY, L, NV>), dim3((unsigned)(wgs < most ? wgs : most)), dim3(T), 0, s,
                               *a);
            return hipGetLastError();
        }
    };
};

template <typename TH, typename TY>
struct Bwd {
    template <int L, int NV>
    struct F {
        static hipError_t call(const BlockArgs* a, const Partition* p, hipStream_t s) {
            constexpr int T = threads_of(L);
            hipLaunchKernelGGL((k_rows_bwd<TH, TY, L, NV>), dim3((unsigned)p->wgs), dim3(T), 0, s, *a, *p,
                               sum_slots(*a), a->ws);
            return hipGetLastError();
        }
    };
};

}  // namespace

bool rows_cover(const BlockArgs& a) { return a.h_cl && a.y_cl && a.C <= 2048 * CG; }

size_t rows_bwd_bytes(const BlockArgs& a) {
    const Partition p = rows_partition(a);
    return (size_t)p.wgs * (p.nsum + p.partials) * a.C * sizeof(float);
}

hipError_t rows_fwd(const BlockArgs& a, int h_bf16, int y_bf16, hipStream_t s) {
    if ((long long)a.B * a.HW == 0) return hipSuccess;
    if (h_bf16 && y_bf16) return for_row<Fwd<bf16_t, bf16_t>::F>(a.C, &a, s);
    if (h_bf16) return for_row<Fwd<bf16_t, float>::F>(a.C, &a, s);
    if (y_bf16) return for_row<Fwd<float, bf16_t>::F>(a.C, &a, s);
    return for_row<Fwd<float, float>::F>(a.C, &a, s);
}

hipError_t rows_bwd(const BlockArgs& a, int h_bf16, int y_bf16, hipStream_t s) {
    const Partition p = rows_partition(a);
    if (p.wgs > 0) {
        hipError_t err;
        if (h_bf16 && y_bf16)
            err = for_row<Bwd<bf16_t, bf16_t>::F>(a.C, &a, &p, s);
        else if (h_bf16)
            err = for_row<Bwd<bf16_t, float>::F>(a.C, &a, &p, s);
        else if (y_bf16)
            err = for_row<Bwd<float, bf16_t>::F>(a.C, &a, &p, s);
        else
            err = for_row<Bwd<float, float>::F>(a.C, &a, &p, s);
        if (err != hipSuccess) return err;
    }
    return block_finalize(a, p, a.ws, s);
}

}  // namespace wtc
