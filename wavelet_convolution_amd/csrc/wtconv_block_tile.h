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
// Where HW is no multiple of PV, or C of eight, the last lane along it moves
// back to end with it and does some of its neighbour's work again: the same
// values to the same addresses. Sums take the elements that two lanes share
// once (kernels of their own, ODD). So a tile needs HW >= PV and C >= 8.
//
// What bounds them (bf16, time of a call on the stream): forwards memory, where
// planes are large (norm 64x96x56x56 15.2 us, 5.1 of the card's 5.2 TB/s;
// residual 32x128x128x128 80 us, 5.0 TB/s), and for small ones the chain of
// latencies: arguments, loads, the sums over channels, stores (residual
// 64x384x14x14 9.6 us, 3.0 TB/s). Backwards the same chain, twice as long, at
// three wavefronts a SIMD (the registers' limit): norm 64x192x28x28 19.7 us (2.9
// TB/s), residual with element dropout 64x96x56x56 54 us (3.6 TB/s), 32x128x128x128
// 164 us (4.1 TB/s); at 29 and 50 vector instructions an element their issue
// alone is 7.0, 24 and 85 us. So what a call does not use is compiled out (X,
// DROP), the rare cases sit behind one branch for the whole patch, and the
// generator's rounds stay a loop over pixels.
#pragma once

#include "wtconv_block_device.h"

namespace wtc {

// v, or zero where element k is one of the `shared` that a neighbour has too.
// ODD: there may be such elements.
template <bool ODD>
__device__ __forceinline__ float once(float v, int k, int shared) {
    if constexpr (ODD) return k < shared ? 0.f : v;
    return v;
}

// A lane's channels: eight from c on, of which the first `shared` are the
// neighbour's too.
template <int CL>
struct Channels {
    int c, shared;
    bool on;
    __device__ __forceinline__ Channels(int C) {
        const int first = (threadIdx.x / 64 * CL + threadIdx.x % CL) * CG;
        on = first < C;
        c = min(first, C - CG);
        shared = on ? first - c : CG;
    }
};

// A lane's pixels in a tile: PV from p on, of which the first `shared` are
// the neighbour's too.
template <int CL, int PV>
struct Pixels {
    static constexpr int PL = 64 / CL, PX = PL * PV;   // pixel lanes, pixels of a tile
    int p, shared;
    bool on;
    __device__ __forceinline__ Pixels(int HW, int tile) {
        const int first = tile * PX + threadIdx.x % 64 / CL * PV;
        on = first < HW;
        p = min(first, HW - PV);
        shared = on ? first - p : PV;
    }
};

// The exchange between wavefronts. Every lane of a wavefront has its sums of
// two values at its PV pixels; they go to one of two buffers in LDS in turn
// (one barrier an exchange). What they come to over all wavefronts is worked
// out once a quad: lane q of four takes pixels q and q + 4, and hands its
// results round by data-parallel moves.
template <int CL, int PV>
struct Exchange {
    static constexpr int PL = 64 / CL, OWN = PV / 4;   // pixels of a lane of the quad
    float* red;                                        // [2 turns][nw][2 values][PL * PV]
    int turn = 0;
    const float* buf;

    __device__ __forceinline__ void put(const float (&a)[PV], const float (&b)[PV]) {
        const int nw = blockDim.x / 64, lane = threadIdx.x % 64, wave = threadIdx.x / 64, pl = lane / CL;
        float* to = red + turn * nw * 2 * PL * PV;
        turn ^= 1;
        if (lane % CL == 0) {
#pragma unroll
            for (int j = 0; j < PV; ++j) {
                to[(wave * 2 * PL + pl) * PV + j] = a[j];
                to[((wave * 2 + 1) * PL + pl) * PV + j] = b[j];
            }
        }
        __syncthreads();
        buf = to + pl * PV + lane % 4;
    }
    // value k (0 or 1) of wavefront w at this lane's i-th pixel of the quad's
    __device__ __forceinline__ float get(int w, int k, int i) const { return buf[(w * 2 + k) * PL * PV + 4 * i]; }
    static __device__ __forceinline__ void round_quad(const float (&own)[OWN], float (&all)[PV]) {
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            all[4 * i] = quad_lane<0>(own[i]);
            all[4 * i + 1] = quad_lane<1>(own[i]);
            all[4 * i + 2] = quad_lane<2>(own[i]);
            all[4 * i + 3] = quad_lane<3>(own[i]);
        }
    }
};

// mean and r of a lane's pixels. Each wavefront takes the mean of its own
// channels and the squares about that mean, and the wavefronts' pairs join
// exactly (Chan, Golub, LeVeque, "Updating formulae and a pairwise algorithm
// for computing sample variances", 1979): sum of squares about the common
// mean = sum over wavefronts of their own + n (their mean - mean)^2. One
// barrier, and no difference of large sums.
template <typename TH, bool HCL, int CL, int PV, bool ODD>
__device__ __forceinline__ void patch_stats(const BlockArgs& a, bool layer, Patch<TH, HCL, PV>& h,
                                            const Channels<CL>& ch, Exchange<CL, PV>& ex, float (&mean)[PV],
                                            float (&r)[PV]) {
    constexpr int WC = CL * CG, OWN = Exchange<CL, PV>::OWN;   // WC: channels of a full wavefront
    const int nw = blockDim.x / 64, wave = threadIdx.x / 64;
    float s[2][PV];
#pragma unroll
    for (int j = 0; j < PV; ++j) s[0][j] = mean[j] = 0.f;
    if (layer) {
        // channels of this wavefront (a scalar: the same for its lanes)
        const float n = (float)min(WC, a.C - __builtin_amdgcn_readfirstlane(wave) * WC);
#pragma unroll
        for (int j = 0; j < PV; ++j) {
#pragma unroll
            for (int i = 0; i < CG; ++i) s[0][j] += once<ODD>(h.at(i, j), i, ch.shared);
        }
        h.renew();
        const float inv = __builtin_amdgcn_rcpf(n);   // a mean near the exact one does
#pragma unroll
        for (int j = 0; j < PV; ++j) {
            s[0][j] = lane_sum<CL>(s[0][j]);
            mean[j] = s[0][j] * inv;
        }
    }
#pragma unroll
    for (int j = 0; j < PV; ++j) {
        s[1][j] = 0.f;
#pragma unroll
        for (int i = 0; i < CG; ++i) {
            const float d = once<ODD>(h.at(i, j) - mean[j], i, ch.shared);
            s[1][j] = fmaf(d, d, s[1][j]);
        }
        s[1][j] = ch.on ? s[1][j] : 0.f;
    }
    h.renew();
#pragma unroll
    for (int j = 0; j < PV; ++j) s[1][j] = lane_sum<CL>(s[1][j]);
    if (nw == 1) {
#pragma unroll
        for (int j = 0; j < PV; ++j) r[j] = rsqrtf(s[1][j] * a.inv_c + a.eps);
        return;
    }
    // a wavefront's squares about the mean that it took, and that mean
    ex.put(mean, s[1]);
    float m[OWN] = {}, q[OWN] = {};
    if (layer) {
#pragma unroll 4
        for (int w = 0; w < nw; ++w) {
            const float part = (float)min(WC, a.C - w * WC) * a.inv_c;
#pragma unroll
            for (int i = 0; i < OWN; ++i) m[i] = fmaf(ex.get(w, 0, i), part, m[i]);
        }
    }
#pragma unroll 4
    for (int w = 0; w < nw; ++w) {
        const float n = (float)min(WC, a.C - w * WC);
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const float d = ex.get(w, 0, i) - m[i];   // zero for rms
            q[i] += fmaf(d * n, d, ex.get(w, 1, i));
        }
    }
#pragma unroll
    for (int i = 0; i < OWN; ++i) q[i] = rsqrtf(q[i] * a.inv_c + a.eps);
    ex.round_quad(m, mean);
    ex.round_quad(q, r);
}

// X: a residual (else a norm alone); DROP: elements are dropped.
template <typename TH, bool HCL, typename TY, bool YCL, int CL, int PV, int MAXT, bool X, bool DROP, bool ODD>
__global__ __launch_bounds__(MAXT) void k_tile_fwd(BlockArgs a, unsigned tiles, unsigned tps) {
    extern __shared__ float red[];
    Exchange<CL, PV> ex{red};
    const Channels<CL> ch(a.C);
    const size_t sh = HCL ? a.C : a.HW, sy = YCL ? a.C : a.HW;
    for (unsigned t = a.near ? xcd_order(blockIdx.x, gridDim.x) : blockIdx.x; t < tiles; t += gridDim.x) {
        const unsigned b = t / tps;
        const Pixels<CL, PV> px(a.HW, (int)(t - b * tps));
        const bool in = !X || a.drop != DROP_SAMPLE || sample_kept(a, (int)b), on = ch.on && px.on;
        const size_t first = (size_t)b * a.C * a.HW;
        const uint32_t planar = (uint32_t)ch.c * a.HW + px.p, rows = (uint32_t)px.p * a.C + ch.c;
        const uint32_t oh = (HCL ? rows : planar) * sizeof(TH), oy = (YCL ? rows : planar) * sizeof(TY);
        Patch<TH, HCL, PV> h;
        Patch<TY, YCL, PV> x;
        // lanes that have nothing of their own read their neighbours' and count
        // zeros; a dropped sample's h is not looked at
        if (in) h.load((const TH*)a.h + first, oh, sh);
        if constexpr (X) x.load((const TY*)a.x + first, oy, sy);
        if (!in || !on) h.zero();
        // y = s x + D'(z wg + bg), with the gate and D's factor in wg and bg
        float wg[CG], bg[CG], xs[CG];
        load_param(a.w, ch.c, 1.f, wg);
        load_param(a.b, ch.c, 0.f, bg);
        if constexpr (X) {
            float g[CG];
            load_param(a.gate_mode == GATE_SAMPLE ? a.gate + (size_t)b * a.C : a.gate, ch.c, 1.f, g);
            load_param(a.xs, ch.c, 1.f, xs);
#pragma unroll
            for (int i = 0; i < CG; ++i) {
                g[i] *= a.keep;
                wg[i] = in ? wg[i] * g[i] : 0.f;
                bg[i] = in ? bg[i] * g[i] : 0.f;
            }
        }
        float mean[PV] = {}, r[PV];
#pragma unroll
        for (int j = 0; j < PV; ++j) r[j] = 1.f;
        if (a.norm != NORM_NONE)
            patch_stats<TH, HCL, CL, PV, ODD>(a, a.norm == NORM_LAYER, h, ch, ex, mean, r);
        if (!on) continue;
        Drops<PV> drop;
        if constexpr (DROP) drop.template draw<ODD>(a, (uint32_t)b * a.HW + px.p, ch.c);
        store_patch<TY, YCL, PV>((TY*)a.y + first, oy, sy, [&](int i, int j) {
            float o = fmaf((h.at(i, j) - mean[j]) * r[j], wg[i], bg[i]);
            if constexpr (DROP) o = drop.kept(o, i, j);
            if constexpr (X) o = fmaf(xs[i], x.at(i, j), o);
            return o;
        });
    }
}

// Over the pixels of one gate (all of them, or a sample's): with e = dy where
// it is kept, S1 = sum e z and S0 = sum e give
//   dw = g k S1, db = g k S0, dg = k (w S1 + b S0)          (k: D's factor),
// so the loop adds two sums, whatever is wanted (X: a residual; else a norm
// alone, whose dw and db they are). With a gate per sample, dw
// and db add up over a workgroup's samples in LDS.
template <typename TH, bool HCL, typename TY, bool YCL, int CL, int PV, int MAXT, bool X, bool DROP, bool ODD>
__global__ __launch_bounds__(MAXT) void k_tile_bwd(BlockArgs a, Partition pt, SumSlots sl, float* slots) {
    extern __shared__ float lds[];
    const Channels<CL> ch(a.C);
    const size_t sh = HCL ? a.C : a.HW, sy = YCL ? a.C : a.HW;
    // with a gate per sample: dw, db [2][lanes' channels], each of its own lane
    const int W = blockDim.x / 64 * CL * CG, own = (threadIdx.x / 64 * CL + threadIdx.x % CL) * CG;
    float* acc = lds + own;
    using EX = Exchange<CL, PV>;
    EX ex{lds + (X && (a.flags & BY_SAMPLE) ? 2 * W : 0)};
    float s1[CG] = {}, s0[CG] = {}, sx[CG] = {};
    const unsigned wg = a.near ? xcd_order(blockIdx.x, gridDim.x) : blockIdx.x;
    float* slot = slots + (size_t)wg * (pt.nsum + pt.partials) * a.C;
    const bool writes = threadIdx.x % 64 < CL && ch.on;   // the lane that writes its channels' sums
    auto pixel_sums = [&](float (&s)[CG]) {
#pragma unroll
        for (int i = 0; i < CG; ++i) s[i] = stride_sum<CL>(s[i]);
    };
    // what a gate's pixels give: dg, and s1 and s0 as parts of dw and db
    auto finish = [&](const float* gate, float* dgp) {
        pixel_sums(s1);
        pixel_sums(s0);
        if (!X || !writes) return;
        float w[CG], bb[CG], g[CG];
        load_param(a.w, ch.c, 1.f, w);
        load_param(a.b, ch.c, 0.f, bb);
        load_param(gate, ch.c, 1.f, g);
#pragma unroll
        for (int i = 0; i < CG; ++i) {
            // without a bias no 0 times S0: where dout is infinite that is no 0
            w[i] = a.keep * (a.b ? fmaf(w[i], s1[i], bb[i] * s0[i]) : w[i] * s1[i]);
            s1[i] *= g[i] * a.keep;
            s0[i] *= g[i] * a.keep;
        }
        if (dgp) store_vec<float, CG>(dgp + ch.c, w);
    };
    if (X && (a.flags & BY_SAMPLE) && writes) {
#pragma unroll
        for (int i = 0; i < CG; ++i) acc[i] = acc[W + i] = 0.f;
    }
    const unsigned tps = (unsigned)pt.tps, t0 = (unsigned)pt.begin(wg), t1 = (unsigned)pt.begin(wg + 1);
    for (unsigned t = t0; t < t1; ++t) {
        uint32_t fl = a.flags;
        asm volatile("" : "+s"(fl));   // tested here, not before the loop
        const unsigned b = t / tps;
        const Pixels<CL, PV> px(a.HW, (int)(t - b * tps));
        const bool in = !X || !(fl & DROPS_SAMPLES) || sample_kept(a, (int)b), on = ch.on && px.on;
        const size_t first = (size_t)b * a.C * a.HW;
        const uint32_t planar = (uint32_t)ch.c * a.HW + px.p, rows = (uint32_t)px.p * a.C + ch.c;
        const uint32_t oh = (HCL ? rows : planar) * sizeof(TH), oy = (YCL ? rows : planar) * sizeof(TY);
        Patch<TH, HCL, PV> h;
        Patch<TY, YCL, PV> d;
        if (in) h.load((const TH*)a.h + first, oh, sh);
        d.load((const TY*)a.dy + first, oy, sy);
        if (!in || !on) h.zero();
        if (!on) d.zero();   // lanes that have nothing of their own count zeros
        if (X && (fl & WANT_DXS) && on) {
            Patch<TY, YCL, PV> x;
            x.load((const TY*)a.x + first, oy, sy);
#pragma unroll
            for (int i = 0; i < CG; ++i)
#pragma unroll
                for (int j = 0; j < PV; ++j)
                    sx[i] = fmaf(once<ODD>(d.at(i, j), j, px.shared), once<ODD>(x.at(i, j), j, px.shared), sx[i]);
            d.renew();
        }
        if (X && (fl & WANT_DX) && on) {
            float xs[CG];
            load_param_if(fl & HAS_XS, a.xs, ch.c, 1.f, xs);
            store_patch<TY, YCL, PV>((TY*)a.dx + first, oy, sy, [&](int i, int j) { return d.at(i, j) * xs[i]; });
        }
        d.renew();
        float mean[PV] = {}, r[PV];
#pragma unroll
        for (int j = 0; j < PV; ++j) r[j] = 1.f;
        if (fl & (LAYER | RMS)) patch_stats<TH, HCL, CL, PV, ODD>(a, fl & LAYER, h, ch, ex, mean, r);
        // from here on d holds e, dy where it is kept
        if (X && !in) d.zero();   // the same for every lane: no gradient passes a dropped sample
        if constexpr (DROP) {
            if (on) {
                Drops<PV> drop;
                drop.template draw<ODD>(a, (uint32_t)b * a.HW + px.p, ch.c);
                d.drop(drop);
                if (!(fl & (LAYER | RMS))) h.drop(drop);   // 0 times NaN is no 0
            }
        }
        auto renew = [&] {
            h.renew();
            d.renew();
        };
        float gw[CG];   // u = e gw
        const float* gate = X ? a.gate + (fl & BY_SAMPLE ? (size_t)b * a.C : 0) : nullptr;
        {
            load_param_if(fl & HAS_W, a.w, ch.c, 1.f, gw);
            if constexpr (X) {
                float g[CG];
                load_param_if(fl & HAS_GATE, gate, ch.c, 1.f, g);
#pragma unroll
                for (int i = 0; i < CG; ++i) gw[i] *= g[i] * a.keep;
            }
        }
        // over pixels, for the channels' gradients, and over channels, for the
        // norm's, without what a neighbour has; z = h r + c, one instruction an
        // element: c's rounding moves z by half a step of mean r, which is what
        // the rounding of the mean itself does
        float ms[2][PV] = {}, c[PV];
#pragma unroll
        for (int j = 0; j < PV; ++j) c[j] = -mean[j] * r[j];
#pragma unroll
        for (int i = 0; i < CG; ++i) {
            const float g = once<ODD>(gw[i], i, ch.shared);
#pragma unroll
            for (int j = 0; j < PV; ++j) {
                const float z = fmaf(h.at(i, j), r[j], c[j]), e = d.at(i, j), u = e * g;
                ms[0][j] += u;
                ms[1][j] = fmaf(u, z, ms[1][j]);
                const float own = once<ODD>(e, j, px.shared);
                s0[i] += own;
                s1[i] = ODD ? s1[i] + once<ODD>(own * z, j, px.shared) : fmaf(own, z, s1[i]);
            }
            // a channel at a time, here and not where the sums are used:
            // fewer values in flight
            asm volatile("" : "+v"(s0[i]), "+v"(s1[i]));
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int j = 0; j < PV; ++j) asm volatile("" : "+v"(ms[0][j]), "+v"(ms[1][j]));
        if (fl & WANT_DH) {
            // dh = r (u - m1 - z m2) = u r + h c2 + c1
            float c1[PV], c2[PV];
            if (fl & (LAYER | RMS)) {
#pragma unroll
                for (int j = 0; j < PV; ++j) {
                    ms[0][j] = lane_sum<CL>(ms[0][j]);
                    ms[1][j] = lane_sum<CL>(ms[1][j]);
                }
                const int nw = blockDim.x / 64;
                if (nw > 1) {
                    ex.put(ms[0], ms[1]);
                    float m1[EX::OWN] = {}, m2[EX::OWN] = {};
#pragma unroll 4
                    for (int w = 0; w < nw; ++w)
#pragma unroll
                        for (int i = 0; i < EX::OWN; ++i) {
                            m1[i] += ex.get(w, 0, i);
                            m2[i] += ex.get(w, 1, i);
                        }
                    ex.round_quad(m1, ms[0]);
                    ex.round_quad(m2, ms[1]);
                }
#pragma unroll
                for (int j = 0; j < PV; ++j) {
                    const float m1 = fl & LAYER ? ms[0][j] * a.inv_c : 0.f, m2 = ms[1][j] * a.inv_c;
                    c2[j] = -r[j] * r[j] * m2;
                    c1[j] = -r[j] * fmaf(c[j], m2, m1);
                }
            } else {
                h.zero();   // dh = u
#pragma unroll
                for (int j = 0; j < PV; ++j) c1[j] = c2[j] = 0.f;
            }
            renew();
            if (on)
                store_patch<TH, HCL, PV>((TH*)a.dh + first, oh, sh, [&](int i, int j) {
                    return fmaf(d.at(i, j) * gw[i], r[j], fmaf(h.at(i, j), c2[j], c1[j]));
                });
        }
        // the last tile of this sample in the workgroup's range
        if (X && (fl & BY_SAMPLE) && (t + 1 == t1 || (t + 1) % tps == 0)) {
            const bool whole = b * tps >= t0 && (b + 1) * tps <= t1;
            finish(gate, !a.dg   ? nullptr
                         : whole ? a.dg + (size_t)b * a.C
                                 : slot + (size_t)(pt.nsum + (b == t0 / tps ? 0 : 1)) * a.C);
            if (writes) {
#pragma unroll
                for (int i = 0; i < CG; ++i) {
                    acc[i] += s1[i];
                    acc[W + i] += s0[i];
                }
            }
#pragma unroll
            for (int i = 0; i < CG; ++i) s1[i] = s0[i] = 0.f;
        }
    }
    if (!X || !(a.flags & BY_SAMPLE)) {
        finish(a.gate, sl.dg >= 0 ? slot + (size_t)sl.dg * a.C : nullptr);
    } else if (writes) {
#pragma unroll
        for (int i = 0; i < CG; ++i) {
            s1[i] = acc[i];
            s0[i] = acc[W + i];
        }
    }
    if (writes && sl.dw >= 0) store_vec<float, CG>(slot + (size_t)sl.dw * a.C + ch.c, s1);
    if (writes && sl.db >= 0) store_vec<float, CG>(slot + (size_t)sl.db * a.C + ch.c, s0);
    if (X && sl.dxs >= 0) {
        pixel_sums(sx);
        if (writes) store_vec<float, CG>(slot + (size_t)sl.dxs * a.C + ch.c, sx);
    }
}

// The shape of a call's tiles.
struct TileShape {
    int cl, pv, nw, px;   // channel lanes, pixels a lane, wavefronts, pixels a tile
    int tps;              // tiles of a sample
};
// Channel lanes: the choice among 4, 8 and 16 with the fewest wavefronts over
// a sample (idle lanes past C and past the plane cost as much as busy ones).
// Sixteen leave 64-byte pieces of a plane and many workgroups of few
// wavefronts, so they need a twentieth fewer (32x128x100x100 residual backward
// at the same number 154 us against 135; 64x384x14x14 at an eighth fewer: norm
// 8.5 against 8.8 forwards, 17.7 against 16.5 backwards). Between four and
// eight at about the same number (one in 64), four have a plane's pieces longer
// and eight fewer wavefronts to a barrier: eight forwards (norm 32x128x127x125
// 57 us against 62, 128x128 57.0 against 56.5; residuals there 87 against 85
// and 81 against 76), four backwards where that is three or four wavefronts
// (residual 208 against 251, 32x128x100x100 124 against 135; 64x64x64x64, two:
// 54.6 against 50.9).
//
// Pixels of a lane: 16 bytes of a plane in bf16 (a tile's fixed costs are
// spread over twice the elements of 8-byte lanes: 32x128x128x128 residual
// forward 81 against 100 us, its backward 163 against 174, the norm's 98
// against 103), unless that leaves less than a wavefront a SIMD, which is all
// latency (64x768x7x7 residual backward 26.0 us with eight pixels, 20.9 with
// four); 4 in fp32, and where more than eight wavefronts share the registers.
//
// cl = 0: fewer channels or pixels than a lane's, more channels than sixteen
// wavefronts hold, a sample of 2^30 elements, or 2^30 tiles.
inline TileShape tile_shape_of(const BlockArgs& a, int pv, bool backward) {
    TileShape best{};
    if (a.C < CG || a.HW < pv) return best;
    // a lane's place in its sample is a 32-bit number of bytes
    if ((uint64_t)a.C * a.HW * sizeof(float) >= 1ull << 32) return best;
    long long least = 0;
    for (int cl : {8, 4, 16}) {
        const int nw = cdiv(a.C, cl * CG);
        if (nw > (cl == 16 ? 16 : 8)) continue;
        const int v = nw > 8 ? 4 : pv, px = 64 / cl * v, tps = cdiv(a.HW, px);
        const long long waves = (long long)nw * tps;
        if ((long long)a.B * tps >= 1ll << 30) continue;   // tiles are counted in 32 bits
        const bool better = cl == 16  ? waves * 21 <= least * 20
                            : cl == 4 ? waves < least || (backward && nw >= 3 && nw <= 4 && waves * 64 <= least * 65)
                                      : waves < least;
        if (best.cl && !better) continue;
        best = TileShape{cl, v, nw, px, tps};
        least = waves;
    }
    return best;
}
inline TileShape tile_shape(const BlockArgs& a, int h_bf16, int y_bf16, bool backward) {
    if (h_bf16 && y_bf16) {
        const TileShape t = tile_shape_of(a, 8, backward);
        if (t.cl && (long long)a.B * t.tps * t.nw >= 4 * 256) return t;
    }
    return tile_shape_of(a, 4, backward);
}

// One file each for the three pairs of memory orders, forwards and backwards.
template <bool HCL, bool YCL>
hipError_t tile_fwd_launch(const BlockArgs& a, int h_bf16, int y_bf16, const TileShape& t, hipStream_t s);
template <bool HCL, bool YCL>
hipError_t tile_bwd_launch(const BlockArgs& a, int h_bf16, int y_bf16, const TileShape& t, const Partition& p,
                           hipStream_t s);

inline size_t tile_lds(const TileShape& t) { return t.nw > 1 ? (size_t)2 * t.nw * 2 * t.px * sizeof(float) : 0; }

// CALL(CL, PV, MAXT) for the shape's channel lanes and wavefronts.
#define WTC_TILE_SHAPES(CALL)                      \
    if (t.cl == 4) return CALL(4, PV, 512);        \
    if (t.cl == 8) return CALL(8, PV, 512);        \
    if (t.nw <= 8) return CALL(16, PV, 512);       \
    return CALL(16, 4, 1024);

template <typename TH, bool HCL, typename TY, bool YCL, int PV, bool X, bool DROP, bool ODD>
hipError_t tile_fwd_odd(const BlockArgs& a, const TileShape& t, hipStream_t s) {
    const unsigned tiles = (unsigned)a.B * (unsigned)t.tps;
    const dim3 grid(tiles < (1u << 21) ? tiles : (1u << 21)), block(64 * t.nw);
#define WTC_CALL(CL, PX, MAXT)                                                                                     \
    [&] {                                                                                                      \
        hipLaunchKernelGGL((k_tile_fwd<TH, HCL, TY, YCL, CL, PX, MAXT, X, DROP, ODD>), grid, block, tile_lds(t), \
                           s, a, tiles, (unsigned)t.tps);                                                      \
        return hipGetLastError();                                                                              \
    }()
    WTC_TILE_SHAPES(WTC_CALL)
#undef WTC_CALL
}

template <typename TH, bool HCL, typename TY, bool YCL, int PV, bool X, bool DROP>
hipError_t tile_fwd_mode(const BlockArgs& a, const TileShape& t, hipStream_t s) {
    if (a.C % CG) return tile_fwd_odd<TH, HCL, TY, YCL, PV, X, DROP, true>(a, t, s);
    return tile_fwd_odd<TH, HCL, TY, YCL, PV, X, DROP, false>(a, t, s);
}

template <typename TH, bool HCL, typename TY, bool YCL, int PV>
hipError_t tile_fwd_typed(const BlockArgs& a, const TileShape& t, hipStream_t s) {
    if (!a.x) return tile_fwd_mode<TH, HCL, TY, YCL, PV, false, false>(a, t, s);
    if (a.drop == DROP_ELEMENT) return tile_fwd_mode<TH, HCL, TY, YCL, PV, true, true>(a, t, s);
    return tile_fwd_mode<TH, HCL, TY, YCL, PV, true, false>(a, t, s);
}

template <typename TH, bool HCL, typename TY, bool YCL, int PV, bool X, bool DROP, bool ODD>
hipError_t tile_bwd_odd(BlockArgs a, const TileShape& t, const Partition& p, hipStream_t s) {
    a.flags = block_flags(a);
    const dim3 grid((unsigned)p.wgs), block(64 * t.nw);
    const size_t lds = tile_lds(t) + (a.gate_mode == GATE_SAMPLE ? sizeof(float) * 2 * t.nw * t.cl * CG : 0);
#define WTC_CALL(CL, PX, MAXT)                                                                                     \
    [&] {                                                                                                      \
        hipLaunchKernelGGL((k_tile_bwd<TH, HCL, TY, YCL, CL, PX, MAXT, X, DROP, ODD>), grid, block, lds, s, a, p, \
                           sum_slots(a), a.ws);                                                                \
        return hipGetLastError();                                                                              \
    }()
    WTC_TILE_SHAPES(WTC_CALL)
#undef WTC_CALL
}

template <typename TH, bool HCL, typename TY, bool YCL, int PV, bool X, bool DROP>
hipError_t tile_bwd_mode(const BlockArgs& a, const TileShape& t, const Partition& p, hipStream_t s) {
    if (a.C % CG || a.HW % t.pv) return tile_bwd_odd<TH, HCL, TY, YCL, PV, X, DROP, true>(a, t, p, s);
    return tile_bwd_odd<TH, HCL, TY, YCL, PV, X, DROP, false>(a, t, p, s);
}

template <typename TH, bool HCL, typename TY, bool YCL, int PV>
hipError_t tile_bwd_typed(const BlockArgs& a, const TileShape& t, const Partition& p, hipStream_t s) {
    if (a.drop == DROP_ELEMENT) return tile_bwd_mode<TH, HCL, TY, YCL, PV, true, true>(a, t, p, s);
    if (block_residual(a))
        return tile_bwd_mode<TH, HCL, TY, YCL, PV, true, false>(a, t, p, s);
    return tile_bwd_mode<TH, HCL, TY, YCL, PV, false, false>(a, t, p, s);
}

// Eight pixels a lane, or four, for bf16 on both sides; four else.
#define WTC_TILE_FWD(HCL, YCL)                                                                                       \
    template <>                                                                                                      \
    hipError_t tile_fwd_launch<HCL, YCL>(const BlockArgs& a, int h_bf16, int y_bf16, const TileShape& t,             \
                                         hipStream_t s) {                                                            \
        if (h_bf16 && y_bf16 && t.pv == 8) return tile_fwd_typed<bf16_t, HCL, bf16_t, YCL, 8>(a, t, s);              \
        if (h_bf16 && y_bf16) return tile_fwd_typed<bf16_t, HCL, bf16_t, YCL, 4>(a, t, s);                           \
        if (h_bf16) return tile_fwd_typed<bf16_t, HCL, float, YCL, 4>(a, t, s);                                      \
        if (y_bf16) return tile_fwd_typed<float, HCL, bf16_t, YCL, 4>(a, t, s);                                      \
        return tile_fwd_typed<float, HCL, float, YCL, 4>(a, t, s);                                                   \
    }

#define WTC_TILE_BWD(HCL, YCL)                                                                                       \
    template <>                                                                                                      \
    hipError_t tile_bwd_launch<HCL, YCL>(const BlockArgs& a, int h_bf16, int y_bf16, const TileShape& t,             \
                                         const Partition& p, hipStream_t s) {                                        \
        if (h_bf16 && y_bf16 && t.pv == 8) return tile_bwd_typed<bf16_t, HCL, bf16_t, YCL, 8>(a, t, p, s);           \
        if (h_bf16 && y_bf16) return tile_bwd_typed<bf16_t, HCL, bf16_t, YCL, 4>(a, t, p, s);                        \
        if (h_bf16) return tile_bwd_typed<bf16_t, HCL, float, YCL, 4>(a, t, p, s);                                   \
        if (y_bf16) return tile_bwd_typed<float, HCL, bf16_t, YCL, 4>(a, t, p, s);                                   \
        return tile_bwd_typed<float, HCL, float, YCL, 4>(a, t, p, s);                                                \
    }

}  // namespace wtc
