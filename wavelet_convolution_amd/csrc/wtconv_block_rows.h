// Block operators on rows: both sides channels last (or tokens). A row of C
// channels is held in the registers of L lanes, NV vectors of eight channels
// a lane, from its one read to its store; the mean, the variance about it and
// the two means of the backward pass are sums over those lanes (within a
// wavefront by data-parallel moves, L > 64 through LDS). A workgroup takes
// several rows at once where L is small, and loops over its rows, so a lane's
// channels never change: parameters are loaded once for its rows where they
// are one vector (NV = 1), and parameter gradients add up in registers, then
// over the workgroup's rows in LDS, then over workgroups in the second stage.
// Forwards memory is the bound (bf16, card's copy rate 5.2 TB/s): norm
// 32,768 x 768 in 21.0 us, 4.8 TB/s; residual into an fp32 stream of that size
// 71.5 us, 4.9. Backwards vector instructions and latency beside it: norm
// 38.6 us, 3.9 TB/s; residual with dropout and a gate per sample,
// 32,768 x 1,024 with an fp32 stream, 72 us, 3.7.
#pragma once

#include "wtconv_block_device.h"

namespace wtc {
namespace {

// Threads of a workgroup: eight wavefronts, so that two fill a CU at the
// kernels' registers and leave few partial sums.
constexpr int threads_of(int L) { return L < 512 ? 512 : L; }

// Where a lane's vectors of eight channels stand. The last vector of a row
// whose C is no multiple of eight (ODD) moves back to end with the row; the
// first `shared` channels of it are its neighbour's too: both do the same work
// on them and store the same values, but sums over a row take them once. Rows
// of fewer than eight channels are one part of a vector (L = 1).
template <int L, int NV, bool ODD>
struct Lanes {
    static constexpr bool PART = L == 1;
    int c[NV], shared[NV];
    bool on[NV];
    int n;   // PART: channels in all
    __device__ __forceinline__ Lanes(int C, int lane) {
        n = C;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int first = (v * L + lane) * CG;
            on[v] = first < C;
            c[v] = PART ? 0 : min(first, C - CG);
            shared[v] = first - c[v];
        }
    }
    // v, where this lane counts channel i of its vector k
    __device__ __forceinline__ float once(float v, int k, int i) const {
        if constexpr (PART) return i < n ? v : 0.f;
        if constexpr (ODD) return i < shared[k] ? 0.f : v;
        return v;
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

// Sums over a row's L lanes, in every lane. L > 64: the wavefronts' sums meet
// in LDS, in one of two buffers in turn (one barrier a sum: a buffer is
// written again only after the barrier of the sum in between).
template <int L>
struct RowSum {
    static constexpr int W = L > 64 ? L / 64 : 1, ALL = threads_of(L) / 64;
    float* red;   // [2 turns][2 values][wavefronts of the workgroup]
    int turn = 0;
    // The two values of each wavefront of this row: the first at [w], the
    // second at [ALL + w].
    __device__ __forceinline__ const float* all(float a, float b) {
        float* buf = red + turn * 2 * ALL;
        turn ^= 1;
        if (threadIdx.x % 64 == 0) {
            buf[threadIdx.x / 64] = a;
            buf[ALL + threadIdx.x / 64] = b;
        }
        __syncthreads();
        return buf + threadIdx.x / L * W;
    }
    __device__ __forceinline__ void two(float& a, float& b) {
        a = lane_sum<(L < 64 ? L : 64)>(a);
        b = lane_sum<(L < 64 ? L : 64)>(b);
        if constexpr (L > 64) {
            const float* buf = all(a, b);
            a = b = 0.f;
#pragma unroll 4
            for (int w = 0; w < W; ++w) {
                a += buf[w];
                b += buf[ALL + w];
            }
        }
    }
};

// mean and r of a row. The variance is the sum of squares about the mean in a
// second sum over the registers; where several wavefronts hold a row, each
// takes it about its own mean and they join exactly (Chan, Golub, LeVeque,
// 1979): one barrier, and no difference of large sums.
template <int L, int NV, bool ODD>
__device__ __forceinline__ void row_stats(const BlockArgs& a, bool layer, const float (&h)[NV][CG],
                                          const Lanes<L, NV, ODD>& at, RowSum<L>& sum, float& mean, float& r) {
    constexpr int N = L < 64 ? L : 64;
    // channels of wavefront w of the row
    auto count = [&](int w) {
        int n = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) n += max(0, min(N * CG, a.C - (v * L + w * N) * CG));
        return (float)n;
    };
    mean = 0.f;
    if (layer) {
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < CG; ++i) s += at.once(h[v][i], v, i);   // zeros past C
        s = lane_sum<N>(s);
        mean = L > 64 ? s / fmaxf(1.f, count(__builtin_amdgcn_readfirstlane(threadIdx.x % L / 64))) : s * a.inv_c;
    }
    float q = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < CG; ++i) {
            const float d = at.on[v] ? at.once(h[v][i] - mean, v, i) : 0.f;
            q = fmaf(d, d, q);
        }
    q = lane_sum<N>(q);
    if constexpr (L > 64) {
        const float* buf = sum.all(mean, q);
        mean = q = 0.f;
#pragma unroll 4
        for (int w = 0; w < RowSum<L>::W; ++w) mean = fmaf(buf[w], count(w) * a.inv_c, mean);
#pragma unroll 4
        for (int w = 0; w < RowSum<L>::W; ++w) {
            const float d = buf[w] - mean;   // zero for rms
            q += fmaf(d * count(w), d, buf[RowSum<L>::ALL + w]);
        }
    }
    r = rsqrtf(q * a.inv_c + a.eps);
}

// Sample of a row (HW rows each).
__device__ __forceinline__ int sample_of(const BlockArgs& a, long long row) {
    return row >> 32 ? (int)(row / a.HW) : (int)((uint32_t)row / (uint32_t)a.HW);
}

// The layouts of a row over lanes, by its vectors of eight channels: the
// fewest lanes that hold it at one vector each, within a wavefront at first,
// then whole workgroups. C = 513 to 1024: two vectors a lane without a barrier,
// but for the backward pass of a residual, which has more to hold and takes
// two wavefronts a row (SPLIT). 32,768 x 768 bf16 norm backward: 36.2 us with
// two vectors, 39.2 with two wavefronts; 8,188 x 1,024 residual backward with
// dropout: 30.7 against 27.7.
template <template <int, int> class F, bool SPLIT, class... A>
auto for_row(int C, A... args) {
    const int vecs = cdiv(C, CG);
    if (vecs <= 1) return F<1, 1>::call(args...);   // the only one for C < 8
    if (vecs <= 4) return F<4, 1>::call(args...);
    if (vecs <= 8) return F<8, 1>::call(args...);
    if (vecs <= 16) return F<16, 1>::call(args...);
    if (vecs <= 32) return F<32, 1>::call(args...);
    if (vecs <= 64) return F<64, 1>::call(args...);
    if (vecs <= 128) return F<SPLIT ? 128 : 64, SPLIT ? 1 : 2>::call(args...);
    if (vecs <= 256) return F<256, 1>::call(args...);
    if (vecs <= 512) return F<512, 1>::call(args...);
    if (vecs <= 1024) return F<1024, 1>::call(args...);
    return F<1024, 2>::call(args...);
}

// K<TH, TY, X, DROP, ODD> for a call: a residual with or without dropped
// elements, or a norm alone; rows with or without a vector that moved back.
template <template <typename, typename, bool, bool, bool> class K, bool SPLIT, typename TH, typename TY, class... A>
hipError_t by_mode(const BlockArgs& a, bool residual, A... args) {
    const bool odd = a.C % CG != 0;
    if (!residual)
        return odd ? for_row<K<TH, TY, false, false, true>::template F, false>(a.C, &a, args...)
                   : for_row<K<TH, TY, false, false, false>::template F, false>(a.C, &a, args...);
    if (a.drop == DROP_ELEMENT)
        return odd ? for_row<K<TH, TY, true, true, true>::template F, SPLIT>(a.C, &a, args...)
                   : for_row<K<TH, TY, true, true, false>::template F, SPLIT>(a.C, &a, args...);
    return odd ? for_row<K<TH, TY, true, false, true>::template F, SPLIT>(a.C, &a, args...)
               : for_row<K<TH, TY, true, false, false>::template F, SPLIT>(a.C, &a, args...);
}
template <template <typename, typename, bool, bool, bool> class K, bool SPLIT, class... A>
hipError_t by_type(const BlockArgs& a, int h_bf16, int y_bf16, bool residual, A... args) {
    if (h_bf16 && y_bf16) return by_mode<K, SPLIT, bf16_t, bf16_t>(a, residual, args...);
    if (h_bf16) return by_mode<K, SPLIT, bf16_t, float>(a, residual, args...);
    if (y_bf16) return by_mode<K, SPLIT, float, bf16_t>(a, residual, args...);
    return by_mode<K, SPLIT, float, float>(a, residual, args...);
}

}  // namespace
}  // namespace wtc
