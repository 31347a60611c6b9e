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

// Where a lane's vectors of eight channels stand. The last vector of a row
// whose C is no multiple of eight moves back to end with the row; `twice`
// names (as drop bits) the channels that it shares with its neighbour: both
// do the same work on them and store the same values, but sums over a row
// take them once. Rows of fewer than eight channels are one part of a vector
// (L = 1).
template <int L, int NV>
struct Lanes {
    static constexpr bool PART = L == 1;
    int c[NV];
    bool on[NV];
    uint32_t twice[NV];
    int n;   // PART: channels in all
    __device__ __forceinline__ Lanes(int C, int lane) {
        n = C;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int first = (v * L + lane) * CG;
            on[v] = first < C;
            c[v] = PART ? 0 : min(first, C - CG);
            twice[v] = PART ? ALL_DROPPED >> min(C, CG) : ALL_DROPPED & ~(ALL_DROPPED >> (first - c[v]));
        }
    }
    template <typename T>
    __device__ __forceinline__ void load(Vec<T, CG>& q, const T* __restrict__ row, int v) const {
        if constexpr (PART)
            q.load_part(row, n);
        else
            q.load(row + c[v]);
    }
    template <typename T>
    __device__ __forceinline__ void store(T* __restrict__ row, const float (&o)[CG], int v) const {
        if constexpr (PART)
            store_part<T, CG>(row, o, n);
        else
            store_vec<T, CG>(row + c[v], o);
    }
    __device__ __forceinline__ void param(const float* p, int v, float none, float (&o)[CG]) const {
        load_param<PART>(p, c[v], none, o, n);
    }
};

// mean and r of a row: the variance about the mean in a second sum over the
// registers (no difference of large sums).
template <typename TH, int NV, int L>
__device__ __forceinline__ void row_stats(const BlockArgs& a, const Vec<TH, CG> (&h)[NV], const Lanes<L, NV>& at,
                                          RowSum<L>& sum, float& mean, float& r) {
    mean = 0.f;
    r = 1.f;
    if (a.norm == NORM_NONE) return;
    const float inv = a.inv_c;
    if (a.norm == NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (at.on[v])
#pragma unroll
                for (int i = 0; i < CG; ++i) s += kept(h[v][i], at.twice[v], i);
        mean = sum.one(s) * inv;
    }
    float q = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
        if (at.on[v])
#pragma unroll
            for (int i = 0; i < CG; ++i) {
                const float d = kept(h[v][i] - mean, at.twice[v], i);
                q = fmaf(d, d, q);
            }
    r = rsqrtf(sum.one(q) * inv + a.eps);
}

template <typename TH, typename TY, int L, int NV>
__global__ __launch_bounds__(threads_of(L)) void k_rows_fwd(BlockArgs a) {
    constexpr int T = threads_of(L), NG = T / L;
    constexpr bool HOIST = NV == 1;
    __shared__ float red[L > 64 ? 4 * L / 64 : 1];
    RowSum<L> sum{red};
    const Lanes<L, NV> at(a.C, threadIdx.x % L);
    const int gi = threadIdx.x / L;
    const long long rows = (long long)a.B * a.HW;
    const uint32_t G = (uint32_t)cdiv(a.C, CG);
    // y = s x + D'(z wg + bg), with the gate and D's factor in wg and bg
    float wg[CG], bg[CG], xs[CG];
    const bool by_sample = a.gate_mode == GATE_SAMPLE;
    auto params = [&](int v, long long bi) {
        float g[CG];
        at.param(a.w, v, 1.f, wg);
        at.param(a.b, v, 0.f, bg);
        at.param(a.xs, v, 1.f, xs);
        at.param(by_sample ? a.gate + bi * a.C : a.gate, v, 1.f, g);
#pragma unroll
        for (int i = 0; i < CG; ++i) {
            g[i] *= a.keep;
            wg[i] *= g[i];
            bg[i] *= g[i];
        }
    };
    if (HOIST && !by_sample && at.on[0]) params(0, 0);
    for (long long r0 = (long long)blockIdx.x * NG; r0 < rows; r0 += (long long)gridDim.x * NG) {
        const long long row = r0 + gi;
        const bool live = row < rows;
        const long long bi = by_sample || a.drop == DROP_SAMPLE ? (live ? row / a.HW : 0) : 0;
        const bool in = live && (a.drop != DROP_SAMPLE || sample_kept(a, (int)bi));
        Vec<TH, CG> h[NV];
        Vec<TY, CG> x[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            h[v].zero();   // a dropped sample's h is not looked at
            if (in && at.on[v]) at.load(h[v], (const TH*)a.h + row * a.C, v);
            if (a.x && live && at.on[v]) at.load(x[v], (const TY*)a.x + row * a.C, v);
        }
        if (HOIST && by_sample && at.on[0]) params(0, bi);
        float mean, r;
        row_stats<TH, NV, L>(a, h, at, sum, mean, r);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (!live || !at.on[v]) continue;
            if constexpr (!HOIST) params(v, bi);
            float o[CG];
#pragma unroll
            for (int i = 0; i < CG; ++i) o[i] = fmaf((h[v][i] - mean) * r, wg[i], bg[i]);
            if (a.drop != DROP_NONE) {
                uint32_t m = in ? 0u : ALL_DROPPED;
                if (a.drop == DROP_ELEMENT)
                    m = drop_bits_at(Philox(a.rng, a.site), (uint32_t)row * G, at.c[v], a.C % CG != 0, a.thr);
#pragma unroll
                for (int i = 0; i < CG; ++i) o[i] = kept(o[i], m, i);
            }
            if (a.x) {
#pragma unroll
                for (int i = 0; i < CG; ++i) o[i] = fmaf(xs[i], x[v][i], o[i]);
            }
            at.store((TY*)a.y + row * a.C, o, v);
        }
    }
}

// Over the rows of one gate (all of them, or a sample's): with e = dy where it
// is kept, S1 = sum e z and S0 = sum e give
//   dw = g k S1, db = g k S0, dg = k (w S1 + b S0)          (k: D's factor),
// so the loop adds two sums, whatever is wanted. Where every row has a gate
// of its own (HW = 1), e holds the gate and dg is written row by row.
template <typename TH, typename TY, int L, int NV>
__global__ __launch_bounds__(threads_of(L)) void k_rows_bwd(BlockArgs a, Partition pt, SumSlots sl, float* slots) {
    constexpr int T = threads_of(L), NG = T / L, W = L * NV * CG;   // W: channels that the lanes hold
    __shared__ float red[L > 64 ? 4 * L / 64 : 1];
    // with a gate per sample: dw, db [2][W]; then, where NG > 1, one sum of each group [NG][W]
    extern __shared__ float lds[];
    RowSum<L> sum{red};
    const int lane = threadIdx.x % L, gi = threadIdx.x / L;
    const Lanes<L, NV> at(a.C, lane);
    const uint32_t G = (uint32_t)cdiv(a.C, CG);
    const bool sample_gate = a.gate_mode == GATE_SAMPLE, by_sample = sample_gate && a.HW > 1;
    const bool each_row = sample_gate && a.HW == 1;
    float *acc = lds, *join = lds + (by_sample ? 2 * W : 0);
    // rows of a sample of the partition (all rows, unless samples count)
    const long long rows = (long long)a.B * a.HW, rps = by_sample ? a.HW : rows;
    float s1[NV][CG] = {}, s0[NV][CG] = {}, sx[NV][CG] = {};
    if (by_sample) {
        for (int e = threadIdx.x; e < 2 * W; e += T) acc[e] = 0.f;
        __syncthreads();
    }
    float* slot = slots + (size_t)blockIdx.x * (pt.nsum + pt.partials) * a.C;
    // sum over the workgroup's groups of lanes, in order; PER channels of it
    // are then a thread's: its own vectors' where NG = 1 (channels that two
    // lanes share are the same in both)
    constexpr int PER = NG > 1 ? cdiv(W, T) : NV * CG;
    auto channel = [&](int q) {   // C: none
        if constexpr (NG > 1) return (int)min((int)threadIdx.x + q * T, a.C);
        return at.on[q / CG] ? at.c[q / CG] + q % CG : a.C;
    };
    auto place = [&](int q) {   // in acc: one for each thread and q
        if constexpr (NG > 1) return (int)threadIdx.x + q * T;
        return (q / CG * L + lane) * CG + q % CG;
    };
    auto joined = [&](const float (&s)[NV][CG], float (&t)[PER]) {
        if constexpr (NG > 1) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (at.on[v])
#pragma unroll
                    for (int i = 0; i < CG; ++i) join[gi * W + at.c[v] + i] = s[v][i];
            __syncthreads();
#pragma unroll
            for (int q = 0; q < PER; ++q) {
                t[q] = 0.f;
                const int e = channel(q);
                if (e < a.C)
#pragma unroll
                    for (int g = 0; g < NG; ++g) t[q] += join[g * W + e];
            }
        } else {
#pragma unroll
            for (int q = 0; q < PER; ++q) t[q] = s[q / CG][q % CG];
        }
    };
    // what a gate's rows give
    auto finish = [&](const float* gate, float* dgp) {
        float t1[PER], t0[PER];
        joined(s1, t1);
        joined(s0, t0);
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int e = channel(q);
            if (e >= a.C) continue;
            if (dgp) dgp[e] = a.keep * ((a.w ? a.w[e] : 1.f) * t1[q] + (a.b ? a.b[e] : 0.f) * t0[q]);
            const float g = (gate ? gate[e] : 1.f) * a.keep;
            if (by_sample) {
                acc[place(q)] += g * t1[q];
                acc[W + place(q)] += g * t0[q];
            } else {
                if (sl.dw >= 0) slot[(size_t)sl.dw * a.C + e] = g * t1[q];
                if (sl.db >= 0) slot[(size_t)sl.db * a.C + e] = g * t0[q];
            }
        }
    };
    const long long t0 = blockIdx.x * pt.per_wg, t1 = min(t0 + pt.per_wg, pt.tiles);
    for (long long t = t0; t < t1; ++t) {
        const long long s = by_sample ? t / pt.tps : 0, r0 = (t - s * pt.tps) * NG + gi, row = s * rps + r0;
        const bool live = r0 < rps;
        const long long bi = by_sample ? s : sample_gate || a.drop == DROP_SAMPLE ? (live ? row / a.HW : 0) : 0;
        const bool in = live && (a.drop != DROP_SAMPLE || sample_kept(a, (int)bi));
        Vec<TH, CG> h[NV];
        Vec<TY, CG> d[NV], x[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            h[v].zero();
            if (in && at.on[v]) at.load(h[v], (const TH*)a.h + row * a.C, v);
            d[v].zero();
            if (live && at.on[v]) at.load(d[v], (const TY*)a.dy + row * a.C, v);
            if (a.dxs && live && at.on[v]) at.load(x[v], (const TY*)a.x + row * a.C, v);
        }
        float mean, r;
        row_stats<TH, NV, L>(a, h, at, sum, mean, r);
        float m1 = 0.f, m2 = 0.f;
        float u[NV][CG];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (!live || !at.on[v]) continue;
            float gw[CG], w[CG], g[CG];
            at.param(a.w, v, 1.f, w);
            at.param(sample_gate ? a.gate + bi * a.C : a.gate, v, 1.f, g);
#pragma unroll
            for (int i = 0; i < CG; ++i) gw[i] = w[i] * g[i] * a.keep;
            uint32_t m = in ? 0u : ALL_DROPPED;
            if (a.drop == DROP_ELEMENT)
                m = drop_bits_at(Philox(a.rng, a.site), (uint32_t)row * G, at.c[v], a.C % CG != 0, a.thr);
            if (each_row && a.dg) {
                float b[CG], o[CG];
                at.param(a.b, v, 0.f, b);
#pragma unroll
                for (int i = 0; i < CG; ++i)
                    o[i] = kept(d[v][i], m, i) * fmaf((h[v][i] - mean) * r, w[i], b[i]) * a.keep;
                at.store(a.dg + row * a.C, o, v);
            }
#pragma unroll
            for (int i = 0; i < CG; ++i) {
                const float z = (h[v][i] - mean) * r, e = kept(d[v][i], m, i);
                const float eg = each_row ? e * g[i] : e;
                s1[v][i] = fmaf(eg, z, s1[v][i]);
                s0[v][i] += eg;
                u[v][i] = e * gw[i];
                const float once = kept(u[v][i], at.twice[v], i);
                m1 += once;
                m2 = fmaf(once, z, m2);
            }
        }
        if (a.norm != NORM_NONE && a.dh) {
            const float inv = a.inv_c;
            sum.two(m1, m2);
            m1 = a.norm == NORM_LAYER ? m1 * inv : 0.f;
            m2 *= inv;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (!live || !at.on[v]) continue;
            if (a.dh) {
                float o[CG];
#pragma unroll
                for (int i = 0; i < CG; ++i) {
                    const float z = (h[v][i] - mean) * r;
                    o[i] = a.norm == NORM_NONE ? u[v][i] : r * (u[v][i] - m1 - z * m2);
                }
                at.store((TH*)a.dh + row * a.C, o, v);
            }
            if (a.dx) {
                float xs[CG], o[CG];
                at.param(a.xs, v, 1.f, xs);
#pragma unroll
                for (int i = 0; i < CG; ++i) o[i] = d[v][i] * xs[i];
                at.store((TY*)a.dx + row * a.C, o, v);
            }
            if (a.dxs) {
#pragma unroll
                for (int i = 0; i < CG; ++i) sx[v][i] = fmaf(d[v][i], x[v][i], sx[v][i]);
            }
        }
        // the last tile of this sample in the workgroup's range
        if (by_sample && (t + 1 == t1 || (t + 1) % pt.tps == 0)) {
            const bool whole = s * pt.tps >= t0 && (s + 1) * pt.tps <= t1;
            finish(a.gate + s * a.C,
                   !a.dg   ? nullptr
                   : whole ? a.dg + s * a.C
                           : slot + (size_t)(pt.nsum + (s == t0 / pt.tps ? 0 : 1)) * a.C);
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < CG; ++i) s1[v][i] = s0[v][i] = 0.f;
        }
    }
    if (by_sample) {   // each thread wrote the places that it reads here
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int e = channel(q);
            if (e >= a.C) continue;
            if (sl.dw >= 0) slot[(size_t)sl.dw * a.C + e] = acc[place(q)];
            if (sl.db >= 0) slot[(size_t)sl.db * a.C + e] = acc[W + place(q)];
        }
    } else {
        finish(each_row ? nullptr : a.gate, sl.dg >= 0 ? slot + (size_t)sl.dg * a.C : nullptr);
    }
    if (sl.dxs >= 0) {
        float tx[PER];
        joined(sx, tx);
#pragma unroll
        for (int q = 0; q < PER; ++q)
            if (channel(q) < a.C) slot[(size_t)sl.dxs * a.C + channel(q)] = tx[q];
    }
}

// The layouts of a row over lanes, by its vectors of eight channels: the
// fewest lanes that hold it at one vector each, then two vectors (C = 513 to
// 1024 stays within a wavefront, without a barrier), then whole workgroups.
template <template <int, int> class F, class... A>
auto for_row(int C, A... args) {
    const int vecs = cdiv(C, CG);
    if (vecs <= 1) return F<1, 1>::call(args...);   // the only one for C < 8
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
    const bool by_sample = a.gate_mode == GATE_SAMPLE && a.HW > 1;
    const long long rows = (long long)a.B * a.HW, rps = by_sample ? a.HW : rows;
    p.tps = (rps + NG - 1) / NG;
    p.tiles = by_sample ? a.B * p.tps : p.tps;
    p.per_wg = (p.tiles + 1023) / 1024;
    if (p.per_wg < 4) p.per_wg = 4;
    p.wgs = (int)((p.tiles + p.per_wg - 1) / p.per_wg);
    p.nsum = sum_slots(a).count;
    p.partials = by_sample && a.dg && p.per_wg % p.tps ? 2 : 0;
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
            constexpr int T = threads_of(L), W = L * NV * CG;
            const bool by_sample = a->gate_mode == GATE_SAMPLE && a->HW > 1;
            const size_t lds = sizeof(float) * ((by_sample ? 2 * W : 0) + (T / L > 1 ? T / L * W : 0));
            hipLaunchKernelGGL((k_rows_bwd<TH, TY, L, NV>), dim3((unsigned)p->wgs), dim3(T), lds, s, *a, *p,
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
