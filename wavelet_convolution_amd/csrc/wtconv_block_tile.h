// Block operators with a planar side: tiles of pixels by channels in registers.
//
// A lane holds PV consecutive pixels of eight consecutive channels. In a
// planar tensor those are eight vectors of PV pixels, in channels-last rows
// PV vectors of eight channels: the change of memory order costs no
// exchange, only another order of use of the same registers. A wavefront is
// CL channel lanes (consecutive lanes, so sums over channels are
// data-parallel moves) by 64 / CL pixel lanes, so both sides move whole
// 64..128-byte pieces of memory per channel or pixel. A workgroup's NW
// wavefronts stand side by side along the channels and cover all of them;
// their sums over channels meet in LDS, one barrier each.
//
// Planes end inside a vector (HW not a multiple of PV): the last pixel lane
// moves back to the plane's last PV pixels and does some of its neighbour's
// work again (the same values to the same addresses); the backward kernel
// leaves those pixels out of its sums.
#pragma once

#include "wtconv_block_device.h"

namespace wtc {

template <typename T, bool CLAST, int PV>
struct Patch {   // [8 channels] x [PV pixels]
    static constexpr int NVEC = CLAST ? PV : CG, LEN = CLAST ? CG : PV;
    Vec<T, LEN> v[NVEC];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < NVEC; ++i) v[i].zero();
    }
    // nc channels and np pixels exist (0: none)
    __device__ __forceinline__ void load(const T* __restrict__ p, size_t step, int nc, int np) {
        const int nv = CLAST ? np : nc, len = CLAST ? nc : np;
#pragma unroll
        for (int i = 0; i < NVEC; ++i) {
            if (i < nv)
                v[i].load(p + i * step, len);
            else
                v[i].zero();
        }
    }
    __device__ __forceinline__ float at(int ch, int px) const { return CLAST ? v[px][ch] : v[ch][px]; }
};

// f(channel, pixel) for every element, rounded and stored.
template <typename T, bool CLAST, int PV, class F>
__device__ __forceinline__ void store_patch(T* __restrict__ p, size_t step, int nc, int np, F&& f) {
    constexpr int NVEC = CLAST ? PV : CG, LEN = CLAST ? CG : PV;
    const int nv = CLAST ? np : nc, len = CLAST ? nc : np;
#pragma unroll
    for (int i = 0; i < NVEC; ++i) {
        if (i >= nv) break;
        float o[LEN];
#pragma unroll
        for (int k = 0; k < LEN; ++k) o[k] = CLAST ? f(k, i) : f(i, k);
        store_vec<T, LEN>(p + i * step, o, len);
    }
}

// Where a lane stands in its tile.
template <int CL, int PV>
struct Place {
    static constexpr int PL = 64 / CL, PX = PL * PV;   // pixel lanes, pixels of a tile
    int c0, nc;      // channels
    int p0, np;      // pixels
    int skip;        // pixels at the front that the neighbour has too
    __device__ __forceinline__ Place(const BlockArgs& a, int tile) {
        const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
        c0 = (wave * CL + lane % CL) * CG;
        nc = max(0, min(CG, a.C - c0));
        p0 = tile * PX + lane / CL * PV;
        np = max(0, min(PV, a.HW - p0));
        skip = 0;
        if (np > 0 && np < PV && a.HW >= PV) {
            skip = PV - np;
            p0 -= skip;
            np = PV;
        }
        if (nc == 0) np = 0;
    }
};

// Sums over all channels of PV pixel values (K sets of them) in every lane.
// The wavefronts' sums go to one of two buffers in turn.
template <int CL, int PV, int K>
__device__ __forceinline__ void channel_sums(float (&s)[K][PV], float* red, int& turn) {
    constexpr int PL = 64 / CL;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < PV; ++j) s[k][j] = lane_sum<CL>(s[k][j]);
    const int nw = blockDim.x / 64;
    if (nw == 1) return;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, pl = lane / CL;
    float* buf = red + (size_t)turn * nw * 2 * PL * PV;
    turn ^= 1;
    if (lane % CL == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < PV; ++j) buf[((wave * K + k) * PL + pl) * PV + j] = s[k][j];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < PV; ++j) s[k][j] = 0.f;
    for (int w = 0; w < nw; ++w)
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < PV; ++j) s[k][j] += buf[((w * K + k) * PL + pl) * PV + j];
}

// mean and r of a lane's pixels.
template <typename TH, bool HCL, int CL, int PV>
__device__ __forceinline__ void patch_stats(const BlockArgs& a, const Patch<TH, HCL, PV>& h, int nc, float* red,
                                            int& turn, float (&mean)[PV], float (&r)[PV]) {
#pragma unroll
    for (int j = 0; j < PV; ++j) {
        mean[j] = 0.f;
        r[j] = 1.f;
    }
    if (a.norm == NORM_NONE) return;
    const float inv = 1.f / (float)a.C;
    float s[1][PV];
    if (a.norm == NORM_LAYER) {
#pragma unroll
        for (int j = 0; j < PV; ++j) {
            s[0][j] = 0.f;
#pragma unroll
            for (int i = 0; i < CG; ++i) s[0][j] += h.at(i, j);   // zeros past C
        }
        channel_sums<CL, PV, 1>(s, red, turn);
#pragma unroll
        for (int j = 0; j < PV; ++j) mean[j] = s[0][j] * inv;
    }
#pragma unroll
    for (int j = 0; j < PV; ++j) {
        s[0][j] = 0.f;
#pragma unroll
        for (int i = 0; i < CG; ++i) {
            const float d = i < nc ? h.at(i, j) - mean[j] : 0.f;
            s[0][j] = fmaf(d, d, s[0][j]);
        }
    }
    channel_sums<CL, PV, 1>(s, red, turn);
#pragma unroll
    for (int j = 0; j < PV; ++j) r[j] = 1.f / sqrtf(s[0][j] * inv + a.eps);
}

// Keep bits of a lane's pixels (eight channels each).
template <int PV>
__device__ __forceinline__ void patch_keep(const BlockArgs& a, long long row0, int c0, bool kept, uint32_t (&m)[PV]) {
    if (a.drop == DROP_ELEMENT) {
        const Philox gen(a.rng, a.site);
        const uint32_t G = (uint32_t)cdiv(a.C, CG), g0 = (uint32_t)row0 * G + (uint32_t)(c0 / CG);
#pragma unroll
        for (int j = 0; j < PV; ++j) m[j] = keep_bits(gen(g0 + j * G), a.thr);
    } else {
#pragma unroll
        for (int j = 0; j < PV; ++j) m[j] = kept ? 0xffu : 0u;
    }
}

template <typename TH, bool HCL, typename TY, bool YCL, int CL, int PV, int MAXT>
__global__ __launch_bounds__(MAXT) void k_tile_fwd(BlockArgs a, long long tiles, int tps) {
    extern __shared__ float red[];
    int turn = 0;
    for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
        const long long b = t / tps;
        const Place<CL, PV> at(a, (int)(t - b * tps));
        const bool kept = a.drop != DROP_SAMPLE || sample_kept(a, (int)b);
        const size_t first = (size_t)b * a.C * a.HW;
        const size_t planar = first + (size_t)at.c0 * a.HW + at.p0, rows = first + (size_t)at.p0 * a.C + at.c0;
        Patch<TH, HCL, PV> h;
        Patch<TY, YCL, PV> x;
        h.load((const TH*)a.h + (HCL ? rows : planar), HCL ? a.C : a.HW, at.nc, kept ? at.np : 0);
        if (a.x) x.load((const TY*)a.x + (YCL ? rows : planar), YCL ? a.C : a.HW, at.nc, at.np);
        float mean[PV], r[PV];
        patch_stats<TH, HCL, CL, PV>(a, h, at.nc, red, turn, mean, r);
        if (at.np <= 0) continue;
        uint32_t m[PV];
        if (a.drop != DROP_NONE) patch_keep<PV>(a, b * a.HW + at.p0, at.c0, kept, m);
        float w[CG], bb[CG], g[CG], xs[CG];
        load_param(a.w, at.c0, at.nc, 1.f, w);
        load_param(a.b, at.c0, at.nc, 0.f, bb);
        load_param(a.gate_mode == GATE_SAMPLE ? a.gate + b * a.C : a.gate, at.c0, at.nc, 1.f, g);
        load_param(a.xs, at.c0, at.nc, 1.f, xs);
        store_patch<TY, YCL, PV>((TY*)a.y + (YCL ? rows : planar), YCL ? a.C : a.HW, at.nc, at.np, [&](int i, int j) {
            float o = (h.at(i, j) - mean[j]) * r[j];
            o = o * w[i] + bb[i];
            if (a.drop != DROP_NONE) o = m[j] >> i & 1 ? o * a.keep : 0.f;
            o *= g[i];
            if (a.x) o = fmaf(xs[i], x.at(i, j), o);
            return o;
        });
    }
}

template <typename TH, bool HCL, typename TY, bool YCL, int CL, int PV, int MAXT>
__global__ __launch_bounds__(MAXT) void k_tile_bwd(BlockArgs a, Partition pt, SumSlots sl, float* slots) {
    extern __shared__ float red[];
    int turn = 0;
    float dw[CG] = {}, db[CG] = {}, dg[CG] = {}, ds[CG] = {};
    float* slot = slots + (size_t)blockIdx.x * (pt.nsum + pt.partials) * a.C;
    const bool sample_gate = a.gate_mode == GATE_SAMPLE, by_sample = a.dg && sample_gate;
    const int lane = threadIdx.x % 64, c0 = (threadIdx.x / 64 * CL + lane % CL) * CG;
    const int nc = max(0, min(CG, a.C - c0));
    // sums over the pixel lanes; a wavefront's channels are its own
    auto put = [&](float (&s)[CG], float* to) {
#pragma unroll
        for (int i = 0; i < CG; ++i) s[i] = stride_sum<CL>(s[i]);
        if (lane < CL && nc > 0) store_vec<float, CG>(to + c0, s, nc);
    };
    const long long t0 = blockIdx.x * pt.per_wg, t1 = min(t0 + pt.per_wg, pt.tiles);
    for (long long t = t0; t < t1; ++t) {
        const long long b = t / pt.tps;
        const Place<CL, PV> at(a, (int)(t - b * pt.tps));
        const bool kept = a.drop != DROP_SAMPLE || sample_kept(a, (int)b);
        const size_t first = (size_t)b * a.C * a.HW;
        const size_t planar = first + (size_t)at.c0 * a.HW + at.p0, rows = first + (size_t)at.p0 * a.C + at.c0;
        const size_t oh = HCL ? rows : planar, oy = YCL ? rows : planar;
        const size_t sh = HCL ? a.C : a.HW, sy = YCL ? a.C : a.HW;
        Patch<TH, HCL, PV> h;
        Patch<TY, YCL, PV> d;
        h.load((const TH*)a.h + oh, sh, at.nc, kept ? at.np : 0);
        d.load((const TY*)a.dy + oy, sy, at.nc, at.np);
        if (a.dxs) {
            Patch<TY, YCL, PV> x;
            x.load((const TY*)a.x + oy, sy, at.nc, at.np);
#pragma unroll
            for (int i = 0; i < CG; ++i)
#pragma unroll
                for (int j = 0; j < PV; ++j) ds[i] = fmaf(j >= at.skip ? d.at(i, j) : 0.f, x.at(i, j), ds[i]);
        }
        if (a.dx && at.np > 0) {
            float xs[CG];
            load_param(a.xs, at.c0, at.nc, 1.f, xs);
            store_patch<TY, YCL, PV>((TY*)a.dx + oy, sy, at.nc, at.np,
                                     [&](int i, int j) { return d.at(i, j) * xs[i]; });
        }
        float mean[PV], r[PV];
        patch_stats<TH, HCL, CL, PV>(a, h, at.nc, red, turn, mean, r);
        uint32_t m[PV];
        patch_keep<PV>(a, b * a.HW + at.p0, at.c0, kept, m);
        float w[CG], bb[CG], g[CG];
        load_param(a.w, at.c0, at.nc, 1.f, w);
        load_param(a.b, at.c0, at.nc, 0.f, bb);
        load_param(sample_gate ? a.gate + b * a.C : a.gate, at.c0, at.nc, 1.f, g);
        float ms[2][PV] = {};
#pragma unroll
        for (int i = 0; i < CG; ++i)
#pragma unroll
            for (int j = 0; j < PV; ++j) {
                // dy is zero past the channels and past the plane
                const bool k = m[j] >> i & 1;
                const float z = (h.at(i, j) - mean[j]) * r[j], di = d.at(i, j);
                const float dv = k ? di * g[i] * a.keep : 0.f, u = dv * w[i];
                ms[0][j] += u;
                ms[1][j] = fmaf(u, z, ms[1][j]);
                const bool own = j >= at.skip;
                const float dvo = own ? dv : 0.f;
                dw[i] = fmaf(dvo, z, dw[i]);
                db[i] += dvo;
                dg[i] = fmaf(own && k ? di : 0.f, fmaf(z, w[i], bb[i]) * a.keep, dg[i]);
            }
        if (a.dh) {
            if (a.norm != NORM_NONE) {
                const float inv = 1.f / (float)a.C;
                channel_sums<CL, PV, 2>(ms, red, turn);
#pragma unroll
                for (int j = 0; j < PV; ++j) {
                    ms[0][j] = a.norm == NORM_LAYER ? ms[0][j] * inv : 0.f;
                    ms[1][j] *= inv;
                }
            }
            // z and u are made again from h and dy rather than kept: an
            // operand that the compiler cannot follow keeps it from holding
            // 16 PV values across the sums
            float keep = a.keep;
#pragma unroll
            for (int j = 0; j < PV; ++j) asm volatile("" : "+v"(mean[j]));
            asm volatile("" : "+v"(keep));
            if (at.np > 0)
                store_patch<TH, HCL, PV>((TH*)a.dh + oh, sh, at.nc, at.np, [&](int i, int j) {
                    const float u = m[j] >> i & 1 ? d.at(i, j) * g[i] * keep * w[i] : 0.f;
                    const float z = (h.at(i, j) - mean[j]) * r[j];
                    return a.norm == NORM_NONE ? u : r[j] * (u - ms[0][j] - z * ms[1][j]);
                });
        }
        // the last tile of this sample in the workgroup's range
        if (by_sample && (t + 1 == t1 || (t + 1) % pt.tps == 0)) {
            const bool whole = b * pt.tps >= t0 && (b + 1) * pt.tps <= t1;
            put(dg, whole ? a.dg + b * a.C : slot + (size_t)(pt.nsum + (b == t0 / pt.tps ? 0 : 1)) * a.C);
#pragma unroll
            for (int i = 0; i < CG; ++i) dg[i] = 0.f;
        }
    }
    if (sl.dw >= 0) put(dw, slot + (size_t)sl.dw * a.C);
    if (sl.db >= 0) put(db, slot + (size_t)sl.db * a.C);
    if (sl.dg >= 0) put(dg, slot + (size_t)sl.dg * a.C);
    if (sl.dxs >= 0) put(ds, slot + (size_t)sl.dxs * a.C);
}

// The shape of a call's tiles.
struct TileShape {
    int cl, pv, nw, px;   // channel lanes, pixels a lane, wavefronts, pixels a tile
    int tps;              // tiles of a sample
};
// Channel lanes: the choice among 4, 8 and 16 with the fewest wavefronts over
// a sample (idle lanes past C and past the plane cost as much as busy ones).
// cl = 0: more channels than sixteen wavefronts hold.
inline TileShape tile_shape(const BlockArgs& a, int pv) {
    TileShape best{};
    long long least = 0;
    for (int cl : {8, 4, 16}) {
        const int nw = cdiv(a.C, cl * CG), px = 64 / cl * pv, tps = cdiv(a.HW, px);
        const long long waves = (long long)nw * tps;
        if (nw > (cl == 16 ? 16 : 8) || (best.cl && waves >= least)) continue;
        best = TileShape{cl, pv, nw, px, tps};
        least = waves;
    }
    return best;
}

#ifndef WTC_PVF
#define WTC_PVF 8
#endif
#ifndef WTC_PVB
#define WTC_PVB 4
#endif
inline int fwd_pv(int h_bf16, int y_bf16) { return h_bf16 && y_bf16 ? WTC_PVF : 4; }
inline int bwd_pv(int h_bf16, int y_bf16) { return h_bf16 && y_bf16 ? WTC_PVB : 4; }

// One file each for the three pairs of memory orders, forwards and backwards.
template <bool HCL, bool YCL>
hipError_t tile_fwd_launch(const BlockArgs& a, int h_bf16, int y_bf16, const TileShape& t, hipStream_t s);
template <bool HCL, bool YCL>
hipError_t tile_bwd_launch(const BlockArgs& a, int h_bf16, int y_bf16, const TileShape& t, const Partition& p,
                           hipStream_t s);

inline size_t tile_lds(const TileShape& t) { return t.nw > 1 ? (size_t)2 * t.nw * 2 * t.px * sizeof(float) : 0; }

// CALL(CL, MAXT) for the shape's channel lanes and wavefronts.
#define WTC_TILE_SHAPES(CALL)                      \
    if (t.cl == 4) return CALL(4, 512);            \
    if (t.cl == 8) return CALL(8, 512);            \
    if (t.nw <= 8) return CALL(16, 512);           \
    return CALL(16, 1024);

template <typename TH, bool HCL, typename TY, bool YCL, int PV>
hipError_t tile_fwd_typed(const BlockArgs& a, const TileShape& t, hipStream_t s) {
    const long long tiles = (long long)a.B * t.tps;
    const dim3 grid((unsigned)(tiles < (1 << 21) ? tiles : (1 << 21))), block(64 * t.nw);
#define WTC_CALL(CL, MAXT)                                                                                          \
    [&] {                                                                                                          \
        hipLaunchKernelGGL((k_tile_fwd<TH, HCL, TY, YCL, CL, PV, MAXT>), grid, block, tile_lds(t), s, a, tiles,    \
                           t.tps);                                                                                 \
        return hipGetLastError();                                                                                  \
    }()
    WTC_TILE_SHAPES(WTC_CALL)
#undef WTC_CALL
}

template <typename TH, bool HCL, typename TY, bool YCL, int PV>
hipError_t tile_bwd_typed(const BlockArgs& a, const TileShape& t, const Partition& p, hipStream_t s) {
    const dim3 grid((unsigned)p.wgs), block(64 * t.nw);
#define WTC_CALL(CL, MAXT)                                                                                          \
    [&] {                                                                                                          \
        hipLaunchKernelGGL((k_tile_bwd<TH, HCL, TY, YCL, CL, PV, MAXT>), grid, block, tile_lds(t), s, a, p,        \
                           sum_slots(a), a.ws);                                                                    \
        return hipGetLastError();                                                                                  \
    }()
    WTC_TILE_SHAPES(WTC_CALL)
#undef WTC_CALL
}

#define WTC_TILE_FWD(HCL, YCL)                                                                                       \
    template <>                                                                                                      \
    hipError_t tile_fwd_launch<HCL, YCL>(const BlockArgs& a, int h_bf16, int y_bf16, const TileShape& t,             \
                                         hipStream_t s) {                                                            \
        if (h_bf16 && y_bf16) return tile_fwd_typed<bf16_t, HCL, bf16_t, YCL, WTC_PVF>(a, t, s);                           \
        if (h_bf16) return tile_fwd_typed<bf16_t, HCL, float, YCL, 4>(a, t, s);                                      \
        if (y_bf16) return tile_fwd_typed<float, HCL, bf16_t, YCL, 4>(a, t, s);                                      \
        return tile_fwd_typed<float, HCL, float, YCL, 4>(a, t, s);                                                   \
    }

#define WTC_TILE_BWD(HCL, YCL)                                                                                       \
    template <>                                                                                                      \
    hipError_t tile_bwd_launch<HCL, YCL>(const BlockArgs& a, int h_bf16, int y_bf16, const TileShape& t,             \
                                         const Partition& p, hipStream_t s) {                                        \
        if (h_bf16 && y_bf16) return tile_bwd_typed<bf16_t, HCL, bf16_t, YCL, WTC_PVB>(a, t, p, s);                        \
        if (h_bf16) return tile_bwd_typed<bf16_t, HCL, float, YCL, 4>(a, t, p, s);                                   \
        if (y_bf16) return tile_bwd_typed<float, HCL, bf16_t, YCL, 4>(a, t, p, s);                                   \
        return tile_bwd_typed<float, HCL, float, YCL, 4>(a, t, p, s);                                                \
    }

}  // namespace wtc
