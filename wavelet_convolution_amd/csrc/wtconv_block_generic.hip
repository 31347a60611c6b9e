// Block operators, generic kernels: any number of channels, any plane, either
// layout on either side. A workgroup takes PX rows (pixels) and 256 / PX
// lanes of each; it reads its rows once for the mean, once for the variance
// and once for the result (from cache where they fit), so nothing limits C.
// The register kernels of the other files serve the sizes that they cover;
// these serve the rest: fewer channels or pixels than a lane's vectors, and
// rows wider than the registers. Latency is most of their time, so the rows
// of a workgroup are as few as leave the wavefronts' loads whole pieces of
// memory.
#include "wtconv_block_device.h"

namespace wtc {
namespace {

constexpr int T = 256;

// The power of two at or below n.
int pow2_below(long long n) {
    int p = 1;
    while (2ll * p <= n && p < T) p *= 2;
    return p;
}

// Rows of a workgroup: neighbouring threads stand on neighbouring rows where a
// side is planar, and on neighbouring channels in rows. Planes: a thread a row
// where there are fewer channels than a group (64x7x56x56 norm forward, bf16:
// 9.3 us, with four lanes a row 12.7); else as many as a sample has, and fewer
// (16 bytes of a plane at least) while that leaves the card empty (4x2500x14x14
// norm forward 56 us, with 64 rows a workgroup 468; 62x347x2x1 7 against 58).
int generic_px(const BlockArgs& a) {
    if (a.h_cl && a.y_cl) return 1;
    if (a.C < CG) return T;
    int px = 64;
    while (px > 8 && (long long)a.B * a.HW / px < 1024) px /= 2;
    return px < a.HW ? px : pow2_below(a.HW);
}

struct At {
    size_t base;
    size_t step;   // between channels
};
__device__ __forceinline__ At at(const BlockArgs& a, int cl, long long row) {
    const long long b = row / a.HW, p = row - b * a.HW;
    return cl ? At{(size_t)row * a.C, 1} : At{(size_t)b * a.C * a.HW + p, (size_t)a.HW};
}

// Sum over the lanes of each row (thread = lane * PX + pixel), by a tree in
// LDS; every lane gets it.
__device__ float row_sum(float v, int px, int PX, float* red) {
    const int t = threadIdx.x;
    __syncthreads();
    red[t] = v;
    for (int n = T / 2; n >= PX; n >>= 1) {
        __syncthreads();
        if (t < n) red[t] += red[t + n];
    }
    __syncthreads();
    return red[px];
}

struct Stats {
    float mean, r;
};
template <typename TH>
__device__ Stats row_stats(const BlockArgs& a, const TH* h, const At& ah, bool live, int lane, int lanes, int px,
                           int PX, float* red) {
    Stats s{0.f, 1.f};
    if (a.norm == NORM_NONE) return s;
    if (a.norm == NORM_LAYER) {
        float sum = 0.f;
        if (live)
#pragma unroll 4
            for (int c = lane; c < a.C; c += lanes) sum += widen(h[ah.base + c * ah.step]);
        s.mean = row_sum(sum, px, PX, red) / (float)a.C;
    }
    float sq = 0.f;
    if (live)
#pragma unroll 4
        for (int c = lane; c < a.C; c += lanes) {
            const float d = widen(h[ah.base + c * ah.step]) - s.mean;
            sq = fmaf(d, d, sq);
        }
    s.r = 1.f / sqrtf(row_sum(sq, px, PX, red) / (float)a.C + a.eps);
    return s;
}

// Drop bits of a row's channels 8 g .. 8 g + 7.
__device__ __forceinline__ uint32_t group_drop(const BlockArgs& a, long long row, int g, bool sample) {
    if (a.drop == DROP_NONE) return 0u;
    if (a.drop == DROP_SAMPLE) return sample ? 0u : ALL_DROPPED;
    const Philox gen(a.rng, a.site);
    const uint32_t G = (uint32_t)cdiv(a.C, CG);
    return drop_bits(gen((uint32_t)row * G + (uint32_t)g), a.thr);
}

template <typename TH, typename TY>
__global__ __launch_bounds__(T) void k_generic_fwd(BlockArgs a, int PX) {
    __shared__ float red[T];
    const TH* h = (const TH*)a.h;
    const TY* x = (const TY*)a.x;
    TY* y = (TY*)a.y;
    const int px = threadIdx.x % PX, lane = threadIdx.x / PX, lanes = T / PX;
    const long long rows = (long long)a.B * a.HW, G = cdiv(a.C, CG);
    for (long long r0 = (long long)blockIdx.x * PX; r0 < rows; r0 += (long long)gridDim.x * PX) {
        const long long row = r0 + px;
        const bool live = row < rows;
        const At ah = at(a, a.h_cl, live ? row : 0), ay = at(a, a.y_cl, live ? row : 0);
        const int b = live ? (int)(row / a.HW) : 0;
        const Stats s = row_stats(a, h, ah, live, lane, lanes, px, PX, red);
        if (!live) continue;
        const bool in = a.drop != DROP_SAMPLE || sample_kept(a, b);
        const float* gate = a.gate ? a.gate + (a.gate_mode == GATE_SAMPLE ? (size_t)b * a.C : 0) : nullptr;
        for (int g = lane; g < G; g += lanes) {
            const uint32_t m = group_drop(a, row, g, in);
            for (int i = 0; i < CG; ++i) {
                const int c = g * CG + i;
                if (c >= a.C) break;
                float v = (widen(h[ah.base + c * ah.step]) - s.mean) * s.r;
                if (a.w) v *= a.w[c];
                if (a.b) v += a.b[c];
                if (gate) v *= gate[c];
                v = kept(v * a.keep, m, i);
                if (x) v += (a.xs ? a.xs[c] : 1.f) * widen(x[ay.base + c * ay.step]);
                y[ay.base + c * ay.step] = narrow_to<TY>(v);
            }
        }
    }
}

// dv and z of one element, from its dy and h.
struct Elem {
    float z, t, dv;
};
__device__ __forceinline__ Elem elem(const BlockArgs& a, const float* gate, const Stats& s, int c, bool keep, float h,
                                     float dy) {
    Elem e;
    e.z = (h - s.mean) * s.r;
    float v = e.z;
    if (a.w) v *= a.w[c];
    if (a.b) v += a.b[c];
    e.t = keep ? v * a.keep : 0.f;
    e.dv = keep ? (gate ? dy * gate[c] : dy) * a.keep : 0.f;
    return e;
}

// dx, dh, and the mean and r of each row for the parameter gradients.
template <typename TH, typename TY>
__global__ __launch_bounds__(T) void k_generic_bwd(BlockArgs a, int PX, float2* stats) {
    __shared__ float red[T];
    const TH* h = (const TH*)a.h;
    const TY* dy = (const TY*)a.dy;
    TH* dh = (TH*)a.dh;
    TY* dx = (TY*)a.dx;
    const int px = threadIdx.x % PX, lane = threadIdx.x / PX, lanes = T / PX;
    const long long rows = (long long)a.B * a.HW, G = cdiv(a.C, CG);
    for (long long r0 = (long long)blockIdx.x * PX; r0 < rows; r0 += (long long)gridDim.x * PX) {
        const long long row = r0 + px;
        const bool live = row < rows;
        const At ah = at(a, a.h_cl, live ? row : 0), ay = at(a, a.y_cl, live ? row : 0);
        const int b = live ? (int)(row / a.HW) : 0;
        const bool in = a.drop != DROP_SAMPLE || sample_kept(a, b);
        const float* gate = a.gate ? a.gate + (a.gate_mode == GATE_SAMPLE ? (size_t)b * a.C : 0) : nullptr;
        Stats s{0.f, 1.f};
        float m1 = 0.f, m2 = 0.f;
        if (a.norm != NORM_NONE) {
            s = row_stats(a, h, ah, live, lane, lanes, px, PX, red);
            if (live && lane == 0) stats[row] = make_float2(s.mean, s.r);
            if (live && in && a.dh)
                for (int g = lane; g < G; g += lanes) {
                    const uint32_t m = group_drop(a, row, g, in);
                    for (int i = 0; i < CG; ++i) {
                        const int c = g * CG + i;
                        if (c >= a.C) break;
                        const Elem e = elem(a, gate, s, c, !(m >> (7 - i) & 1), widen(h[ah.base + c * ah.step]),
                                            widen(dy[ay.base + c * ay.step]));
                        const float u = a.w ? e.dv * a.w[c] : e.dv;
                        m1 += u;
                        m2 = fmaf(u, e.z, m2);
                    }
                }
            m1 = a.norm == NORM_LAYER ? row_sum(m1, px, PX, red) / (float)a.C : 0.f;
            m2 = row_sum(m2, px, PX, red) / (float)a.C;
        }
        if (!live) continue;
        for (int g = lane; g < G; g += lanes) {
            const uint32_t m = group_drop(a, row, g, in);
            for (int i = 0; i < CG; ++i) {
                const int c = g * CG + i;
                if (c >= a.C) break;
                const float d = widen(dy[ay.base + c * ay.step]);
                if (dx) dx[ay.base + c * ay.step] = narrow_to<TY>(a.xs ? d * a.xs[c] : d);
                if (!dh) continue;
                float o = 0.f;   // a dropped sample's h is not looked at
                if (in) {
                    const float hv = a.norm != NORM_NONE ? widen(h[ah.base + c * ah.step]) : 0.f;
                    const Elem e = elem(a, gate, s, c, !(m >> (7 - i) & 1), hv, d);
                    const float u = a.w ? e.dv * a.w[c] : e.dv;
                    o = a.norm == NORM_NONE ? u : s.r * (u - m1 - e.z * m2);
                }
                dh[ah.base + c * ah.step] = narrow_to<TH>(o);
            }
        }
    }
}

// Parameter gradients: a thread owns the eight channels of one group and adds
// every RL-th row of its workgroup's range (a tile is one row here); the RL
// threads of a group join in LDS, in a fixed order.
template <typename TH, typename TY>
__global__ __launch_bounds__(T) void k_generic_grads(BlockArgs a, const float2* stats, Partition pt, SumSlots sl,
                                                     float* slots, int RL) {
    __shared__ float red[T][CG + 1];   // an odd step: no two lanes on one bank
    const TH* h = (const TH*)a.h;
    const TY* x = (const TY*)a.x;
    const TY* dy = (const TY*)a.dy;
    const int t = threadIdx.x, ri = t % RL;
    const int g = blockIdx.x * (T / RL) + t / RL, c0 = g * CG, n = min(CG, a.C - c0);   // n <= 0: no such group
    const bool writes = ri == 0 && n > 0;
    float* slot = slots + (size_t)blockIdx.y * (pt.nsum + pt.partials) * a.C;
    float dw[CG] = {}, db[CG] = {}, dg[CG] = {}, ds[CG] = {};
    const long long t0 = pt.begin(blockIdx.y), t1 = pt.begin(blockIdx.y + 1);
    const bool by_sample = a.dg && a.gate_mode == GATE_SAMPLE;
    // the sum over the rows' threads, stored by one of them
    auto store = [&](const float (&v)[CG], float* to) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < CG; ++i) red[t][i] = v[i];
        for (int k = RL / 2; k > 0; k /= 2) {
            __syncthreads();
            if (ri < k)
#pragma unroll
                for (int i = 0; i < CG; ++i) red[t][i] += red[t + k][i];
        }
        if (!writes) return;
#pragma unroll
        for (int i = 0; i < CG; ++i)
            if (i < n) to[c0 + i] = red[t][i];
    };
    for (long long from = t0; from < t1;) {
        // the rows of one sample in the range, where samples count, else all
        const long long b0 = from / pt.tps, to = by_sample ? min(t1, (b0 + 1) * pt.tps) : t1;
        for (long long row = from + ri; row < to; row += RL) {
            const int b = (int)(row / a.HW);
            const At ah = at(a, a.h_cl, row), ay = at(a, a.y_cl, row);
            const bool in = a.drop != DROP_SAMPLE || sample_kept(a, b);
            const uint32_t m = n > 0 ? group_drop(a, row, g, in) : 0u;
            const float* gate = a.gate ? a.gate + (a.gate_mode == GATE_SAMPLE ? (size_t)b * a.C : 0) : nullptr;
            Stats s{0.f, 1.f};
            if (a.norm != NORM_NONE) s = Stats{stats[row].x, stats[row].y};
#pragma unroll
            for (int i = 0; i < CG; ++i) {
                if (i >= n) break;
                const int c = c0 + i;
                const float d = widen(dy[ay.base + c * ay.step]);
                if (a.dxs) ds[i] = fmaf(d, widen(x[ay.base + c * ay.step]), ds[i]);
                if (in && a.h) {
                    const Elem e = elem(a, gate, s, c, !(m >> (7 - i) & 1), widen(h[ah.base + c * ah.step]), d);
                    dw[i] = fmaf(e.dv, e.z, dw[i]);
                    db[i] += e.dv;
                    dg[i] = fmaf(d, e.t, dg[i]);
                }
            }
        }
        if (by_sample) {
            const bool whole = b0 * pt.tps >= t0 && (b0 + 1) * pt.tps <= t1;
            store(dg, whole ? a.dg + (size_t)b0 * a.C
                            : slot + (size_t)(pt.nsum + (b0 == t0 / pt.tps ? 0 : 1)) * a.C);
#pragma unroll
            for (int i = 0; i < CG; ++i) dg[i] = 0.f;
        }
        from = to;
    }
    if (sl.dw >= 0) store(dw, slot + (size_t)sl.dw * a.C);
    if (sl.db >= 0) store(db, slot + (size_t)sl.db * a.C);
    if (sl.dg >= 0) store(dg, slot + (size_t)sl.dg * a.C);
    if (sl.dxs >= 0) store(ds, slot + (size_t)sl.dxs * a.C);
}

// Second stage. A workgroup takes 16 channels of one sum: a lane adds four
// channels (16 bytes) of the slots k = l, l + 256, ..., data-parallel moves
// join a wavefront's 16 lanes of the same channels, and LDS the 16
// wavefronts, all in a fixed order. Latency is all of its time, so its loads
// are few, wide and in flight together, with one barrier after them. Blocks
// past the channel sums join the partial gate gradients of one sample each,
// over the workgroups that its tiles lie in.
constexpr int FC = 16, FT = 1024, FL = FT * 4 / FC;
__global__ __launch_bounds__(FT) void k_finalize(BlockArgs a, Partition pt, SumSlots sl, const float* slots,
                                                 int cblocks) {
    __shared__ float red[FT / 64][FC];
    const int quad = threadIdx.x % (FC / 4), lane = threadIdx.x / (FC / 4);
    const size_t slot = (size_t)(pt.nsum + pt.partials) * a.C;
    const long long items = (long long)cblocks * (pt.nsum + (pt.partials ? a.B : 0));
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
        const long long what = item / cblocks;
        const int c0 = (int)(item - what * cblocks) * FC, c = c0 + quad * 4;
        float* dst;
        float sum[4] = {};
        auto add = [&](const float* p) {
            if (c + 4 <= a.C) {
                Vec<float, 4> v;
                v.load(p + c);
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[i] += v[i];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + i < a.C) sum[i] += p[c + i];
            }
        };
        if (what < pt.nsum) {
            dst = what == sl.dw ? a.dw : what == sl.db ? a.db : what == sl.dg ? a.dg : a.dxs;
#pragma unroll 4
            for (int k = lane; k < pt.wgs; k += FL) add(slots + k * slot + what * a.C);
        } else {
            const long long b = what - pt.nsum, k0 = pt.owner(b * pt.tps), k1 = pt.owner((b + 1) * pt.tps - 1);
            if (k0 == k1) continue;   // written by its one workgroup (the same for the whole block)
            dst = a.dg + b * a.C;
            for (long long k = k0 + lane; k <= k1; k += FL)
                add(slots + k * slot + (size_t)(pt.nsum + (pt.begin(k) / pt.tps == b ? 0 : 1)) * a.C);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = stride_sum<4>(sum[i]);
        if (threadIdx.x % 64 < 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) red[threadIdx.x / 64][quad * 4 + i] = sum[i];
        }
        __syncthreads();
        if (threadIdx.x < FC && c0 + (int)threadIdx.x < a.C) {
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < FT / 64; ++w) t += red[w][threadIdx.x];
            dst[c0 + threadIdx.x] = t;
        }
        __syncthreads();
    }
}

// Threads that share a group of the parameter gradients: neighbouring rows of
// a plane (a sample's, where samples count), and what the groups leave over.
int grads_rl(const BlockArgs& a) {
    const int most = a.gate_mode == GATE_SAMPLE ? pow2_below(a.HW) : T;
    int rl = a.h_cl && a.y_cl ? 1 : min(64, pow2_below(a.HW));
    while (rl < most && rl * cdiv(a.C, CG) <= T / 2) rl *= 2;
    return rl < most ? rl : most;
}

// One row a tile; each thread takes a few rows, so that a workgroup's slot
// (nsum rows of its own) is little beside what it reads.
Partition generic_partition(const BlockArgs& a) {
    Partition p{};
    const bool sample = a.gate_mode == GATE_SAMPLE;
    p.tiles = (long long)a.B * a.HW;
    p.tps = a.dg && sample ? a.HW : p.tiles;
    const int rl = grads_rl(a), per = max(8, sample ? rl : 2 * rl);
    p.wgs = (int)min(1024ll, (p.tiles + per - 1) / per);
    p.nsum = sum_slots(a).count;
    p.partials = a.dg && sample ? 2 : 0;
    return p;
}

size_t slots_bytes(const BlockArgs& a, const Partition& p) {
    return (size_t)p.wgs * (p.nsum + p.partials) * a.C * sizeof(float);
}

size_t stats_bytes(const BlockArgs& a) {
    return a.norm == NORM_NONE ? 0 : ((size_t)a.B * a.HW * sizeof(float2) + 255) / 256 * 256;
}

// Workgroups for n items; the kernels loop over what is left.
unsigned grid_of(long long n) { return (unsigned)(n < (1 << 20) ? n : (1 << 20)); }

}  // namespace

hipError_t block_finalize(const BlockArgs& a, const Partition& p, const float* slots, hipStream_t s) {
    const int cblocks = cdiv(a.C, FC);
    const long long items = (long long)cblocks * (p.nsum + (p.partials ? a.B : 0));
    if (items == 0) return hipSuccess;
    hipLaunchKernelGGL(k_finalize, dim3(grid_of(items)), dim3(FT), 0, s, a, p, sum_slots(a), slots, cblocks);
    return hipGetLastError();
}

size_t block_generic_bwd_bytes(const BlockArgs& a) { return stats_bytes(a) + slots_bytes(a, generic_partition(a)); }

#define WTC_TYPES(KERNEL, GRID, ...)                                                                       \
    do {                                                                                                   \
        if (h_bf16 && y_bf16)                                                                              \
            hipLaunchKernelGGL((KERNEL<bf16_t, bf16_t>), GRID, dim3(T), 0, s, __VA_ARGS__);                \
        else if (h_bf16)                                                                                   \
            hipLaunchKernelGGL((KERNEL<bf16_t, float>), GRID, dim3(T), 0, s, __VA_ARGS__);                 \
        else if (y_bf16)                                                                                   \
            hipLaunchKernelGGL((KERNEL<float, bf16_t>), GRID, dim3(T), 0, s, __VA_ARGS__);                 \
        else                                                                                               \
            hipLaunchKernelGGL((KERNEL<float, float>), GRID, dim3(T), 0, s, __VA_ARGS__);                  \
    } while (0)

hipError_t block_generic_fwd(const BlockArgs& a, int h_bf16, int y_bf16, hipStream_t s) {
    const int PX = generic_px(a);
    const long long rows = (long long)a.B * a.HW;
    if (rows == 0) return hipSuccess;
    WTC_TYPES(k_generic_fwd, dim3(grid_of((rows + PX - 1) / PX)), a, PX);
    return hipGetLastError();
}

hipError_t block_generic_bwd(const BlockArgs& a, int h_bf16, int y_bf16, hipStream_t s) {
    const int PX = generic_px(a);
    const long long rows = (long long)a.B * a.HW;
    float2* stats = (float2*)a.ws;
    if (rows > 0) {
        WTC_TYPES(k_generic_bwd, dim3(grid_of((rows + PX - 1) / PX)), a, PX, stats);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    const Partition p = generic_partition(a);
    float* slots = (float*)((char*)a.ws + stats_bytes(a));
    const SumSlots sl = sum_slots(a);
    if (p.wgs > 0 && (sl.count || (a.dg && a.gate_mode == GATE_SAMPLE))) {
        const int rl = grads_rl(a);
        WTC_TYPES(k_generic_grads, dim3((unsigned)cdiv(cdiv(a.C, CG), T / rl), (unsigned)p.wgs), a, stats, p, sl, slots,
                  rl);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return block_finalize(a, p, slots, s);
}

}  // namespace wtc
