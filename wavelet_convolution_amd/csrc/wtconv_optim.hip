// AdamW and the gradients' norm over many tensors. Memory is the bound: every
// element of a parameter, its gradient and its states is read once and
// written once (the card copies at 5.2 TB/s; a large tensor multiplied in place
// reaches 6.0). AdamW: 34.6 M bf16 parameters in 330 tensors with fp32 master
// copies, 28 bytes an element, 189 us, 5.1 TB/s; 76 M with states in 8 bits, 16
// bytes an element, 212 us, 5.8 TB/s. Norm: 34.6 M bf16 elements 18.2 us, of which
// 6 are the latency of its two launches.
#include "wtconv_block_device.h"
#include "wtconv_optim.h"

namespace wtc {
namespace {

constexpr int T = 256;

// The tensor of a workgroup: the last one whose first workgroup is not behind
// it. All lanes look at a first workgroup each, and a ballot counts.
__device__ __forceinline__ uint32_t first_wg(const AdamTensor& t) { return t.wg; }
__device__ __forceinline__ uint32_t first_wg(const NormTensor& t) { return t.w[2] >> 18; }
template <class A>
__device__ __forceinline__ int tensor_of(const A& a, uint32_t wg) {
    constexpr int N = (A::MOST + 63) / 64;   // loads that are in flight together
    const int lane = threadIdx.x % 64;
    uint32_t at[N];
#pragma unroll
    for (int i = 0; i < N; ++i) at[i] = i * 64 < a.n ? first_wg(a.t[min(i * 64 + lane, a.n - 1)]) : 0;
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += (int)__popcll(__ballot(i * 64 + lane < a.n && at[i] <= wg));
    return __builtin_amdgcn_readfirstlane(n - 1);
}

// Largest of 64 lanes, for values that are not negative: as whole numbers,
// where a NaN is the largest.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0u, v, CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float wave_max(uint32_t v) {
    v = dpp_max<0xB1>(v);
    v = dpp_max<0x4E>(v);
    v = dpp_max<0x141>(v);
    v = dpp_max<0x140>(v);
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(r[0], r[1]);
    const auto q = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return __uint_as_float(max(q[0], q[1]));
}

// Four e4m3 numbers from |q| <= 448 (a little more by rounding), to nearest.
__device__ __forceinline__ uint32_t e4m3_near(const float (&q)[4]) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
}
// One, up or down by 16 bits u. Times 2^-120 a float has e4m3's exponent (its
// subnormals too) and 20 bits more of fraction: the carry of the random bits
// out of those 20 rounds up.
__device__ __forceinline__ uint32_t e4m3_random(float q, uint32_t u) {
    float f = fabsf(q);
    f = f > 448.f ? 448.f : f;   // a NaN stays
    const uint32_t code = min((__float_as_uint(f * 0x1p-120f) + (u << 4) + 8) >> 20, 0x7fu);
    return code | (__float_as_uint(q) >> 24 & 0x80u);
}
__device__ __forceinline__ void widen_e4m3(uint32_t w, float unit, float (&o)[4]) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    o[0] = lo[0] * unit;
    o[1] = lo[1] * unit;
    o[2] = hi[0] * unit;
    o[3] = hi[1] * unit;
}

// 1 - e^x for x <= 0: the series of e^x - 1 down to -1 (its next term, x^12 / 12!,
// is 2^-28 of the sum there), so that no near numbers are subtracted; below, the
// power itself.
__device__ __forceinline__ float one_less_exp(float x) {
    constexpr float inv[] = {1.f, 1.f / 2, 1.f / 6, 1.f / 24, 1.f / 120, 1.f / 720, 1.f / 5040, 1.f / 40320, 1.f / 362880,
                             1.f / 3628800, 1.f / 39916800};
    float s = inv[10];
#pragma unroll
    for (int k = 9; k >= 0; --k) s = fmaf(s, x, inv[k]);
    return x > -1.f ? -x * s : 1.f - __builtin_amdgcn_exp2f(x * 1.44269504f);
}

// The square root to one step, by the hardware's instruction where it has the
// range (a denormal would be zero there, and a moment divided by eps alone).
__device__ __forceinline__ void roots(const float (&v)[4], float (&root)[4]) {
    uint32_t low = ~0u;   // of those that are not zero
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        root[i] = __builtin_amdgcn_sqrtf(v[i]);
        low = min(low, __float_as_uint(v[i]) - 1);
    }
    if (low < __float_as_uint(0x1p-100f)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) root[i] = sqrtf(v[i]);
    }
}

// A wavefront takes one block of 256 elements, a lane four of them, and ends:
// the next one's loads are on their way while it computes, with more of them in
// flight than a loop over blocks keeps (four blocks a wavefront, two at a time,
// measured before the arithmetic below had its present form: 219 us for 190, with
// states in 8 bits 250 for 233, now 212; streaming stores changed neither). It
// takes two where an element is only ten or twelve bytes and its instructions are
// the bound, one after the other: 33 M bf16 parameters without master copies,
// states in 8 bits, 67 us for 77, with random rounding 84 for 91; fp32 parameters
// 107 for 99.
template <typename P, typename G, bool MASTER, int MODE, int TENSORS>
__global__ __launch_bounds__(T) void k_adamw(AdamTable<TENSORS> a, uint32_t wgs) {
    const float f = a.factor ? *a.factor : 1.f;
    if (!(fabsf(f) < INFINITY)) return;
    const uint32_t wg = blockIdx.y * gridDim.x + blockIdx.x;
    if (wg >= wgs) return;
    const AdamTensor& t = a.t[tensor_of(a, wg)];
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    constexpr int BLOCKS = adam_blocks(sizeof(P) == 2, MASTER, MODE);
    const uint64_t count = ((uint64_t)(t.more >> 30) << 32 | t.last) + 1;
    const uint32_t number = t.more & (ADAM_NUMBERS - 1), of = t.more >> 26 & (ADAM_RATES - 1);
    float rate = 0.f, root_scale = 0.f, decay = 0.f;
#pragma unroll 1
    for (int b = 0; b < BLOCKS; ++b) {
        const uint64_t first = ((uint64_t)(wg - t.wg) * (T / 64) * BLOCKS + b * (T / 64) + wave) * OB;
        if (first >= count) return;
        // a lane's n elements of the tensor from e on, and its place in the states
        const bool full = count - first >= OB;   // the same for every lane
        const uint64_t e = first + 4 * lane;
        const int n = full ? 4 : e >= count ? 0 : count - e < 4 ? (int)(count - e) : 4;
        const size_t block = t.block + first / OB, s = block * OB + 4 * lane;
        P* const param = (P*)t.p + first;
        const G* const grad = (const G*)t.g + first;
        Vec<P, 4> pv;
        Vec<float, 4> xv, mv, vv;
        Vec<G, 4> gv;
        uint32_t m8 = 0, v8 = 0;
        float2 unit = make_float2(0.f, 0.f);
        if (full) {
            gv.load(grad + 4 * lane);
            if constexpr (!MASTER) pv.load(param + 4 * lane);
        } else {
            gv.load_part(grad + 4 * lane, n);
            if constexpr (!MASTER) pv.load_part(param + 4 * lane, n);
        }
        if constexpr (MASTER) xv.load(a.master + s);
        if constexpr (MODE == STATES_32) {
            mv.load((const float*)a.m + s);
            vv.load((const float*)a.v + s);
        } else {
            m8 = *(const uint32_t*)((const char*)a.m + s);
            v8 = *(const uint32_t*)((const char*)a.v + s);
            unit = ((const float2*)a.scales)[block];
        }
        if (b == 0) {
            // 1 / sqrt(1 - beta^t) of the first beta in the lower lanes, of the
            // second in the upper ones
            const float half = __builtin_amdgcn_rsqf(one_less_exp((float)max(1ll, *a.step) * (lane < 32 ? a.log1 : a.log2)));
            const float half1 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(half), 0));
            root_scale = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(half), 32));
            const float lr = a.lr_factor ? a.lr[of] * *a.lr_factor : a.lr[of];
            decay = 1.f - lr * a.wd[of];
            rate = lr * half1 * half1;
        }
        float m[4], v[4], x[4], root[4];
        if constexpr (MODE == STATES_32) {
#pragma unroll
            for (int i = 0; i < 4; ++i) m[i] = mv[i], v[i] = vv[i];
        } else {
            widen_e4m3(m8, unit.x, m);
            widen_e4m3(v8, unit.y, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] *= v[i];
            if (!full) {   // nothing past the tensor's end
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i >= n) m[i] = v[i] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float g = gv[i] * f;
            m[i] = fmaf(a.b1, m[i], a.a1 * g);
            v[i] = fmaf(a.b2, v[i], a.a2 * g * g);
        }
        roots(v, root);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (MASTER)
                x[i] = xv[i];
            else
                x[i] = pv[i];
            x[i] = fmaf(-rate * m[i], __builtin_amdgcn_rcpf(fmaf(root[i], root_scale, a.eps)), x[i] * decay);
        }
        if (full) {
            store_vec<P, 4>(param + 4 * lane, x);
            if constexpr (MASTER) store_vec<float, 4>(a.master + s, x);
        } else {
            store_part<P, 4>(param + 4 * lane, x, n);
            if constexpr (MASTER) store_part<float, 4>(a.master + s, x, n);
        }
        if constexpr (MODE == STATES_32) {
            if (full) {
                store_vec<float, 4>((float*)a.m + s, m);
                store_vec<float, 4>((float*)a.v + s, v);
            } else {
                store_part<float, 4>((float*)a.m + s, m, n);
                store_part<float, 4>((float*)a.v + s, v, n);
            }
        } else {
            uint32_t top = 0, most = 0;   // as whole numbers, as in the wavefront's
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                top = max(top, __float_as_uint(m[i]) & 0x7fffffffu);
                most = max(most, __float_as_uint(root[i]));
            }
            // a moment below 2^-100 is none; a root is above 2^-75 or zero
            float um = wave_max(top), uv = wave_max(most);
            um = um < 0x1p-100f ? 0.f : um * (1.f / 448.f);
            uv *= 1.f / 448.f;
            const float per_m = um == 0.f ? 0.f : __builtin_amdgcn_rcpf(um), per_v = uv == 0.f ? 0.f : __builtin_amdgcn_rcpf(uv);
            float q[4], r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                q[i] = m[i] * per_m;
                // 2^-9 at least, but for zero: a root times 2^100 is more than that
                r[i] = root[i] * per_v;
                const float least = fminf(root[i] * 0x1p100f, 0x1p-9f);
                r[i] = r[i] < least ? least : r[i];
            }
            uint32_t cm, cv;
            if constexpr (MODE == STATES_8) {
                cm = e4m3_near(q);
                cv = e4m3_near(r);
            } else {
                const uint4 bits = Philox(a.rng, a.site + number)((uint32_t)(e / 4));
                const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
                cm = cv = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    cm |= e4m3_random(q[i], w[i] & 0xffffu) << (8 * i);
                    cv |= e4m3_random(r[i], w[i] >> 16) << (8 * i);
                }
            }
            *(uint32_t*)((char*)a.m + s) = cm;
            *(uint32_t*)((char*)a.v + s) = cv;
            if (lane == 0) ((float2*)a.scales)[block] = make_float2(um, uv);
        }
    }
}

// The same arguments with a shorter table.
template <class Head, class Table, class A>
Table shorter(const A& a) {
    Table b;
    (Head&)b = a;
    for (int i = 0; i < a.n; ++i) b.t[i] = a.t[i];
    return b;
}

template <typename P, typename G, bool MASTER, int MODE>
hipError_t adamw_by_count(const AdamArgs& a, uint32_t wgs, hipStream_t s) {
    // a grid's side has fewer than 2^32 lanes
    const uint32_t x = wgs < 1u << 20 ? wgs : 1u << 20;
    const dim3 grid(x, (wgs + x - 1) / x);
    if (a.n <= ADAM_FEW)
        hipLaunchKernelGGL((k_adamw<P, G, MASTER, MODE, ADAM_FEW>), grid, dim3(T), 0, s,
                           (shorter<AdamHead, AdamTable<ADAM_FEW>>(a)), wgs);
    else
        hipLaunchKernelGGL((k_adamw<P, G, MASTER, MODE, ADAM_TENSORS>), grid, dim3(T), 0, s, a, wgs);
    return hipGetLastError();
}
template <typename P, typename G, bool MASTER>
hipError_t adamw_by_mode(const AdamArgs& a, uint32_t wgs, int mode, hipStream_t s) {
    if (mode == STATES_32) return adamw_by_count<P, G, MASTER, STATES_32>(a, wgs, s);
    return mode == STATES_8 ? adamw_by_count<P, G, MASTER, STATES_8>(a, wgs, s)
                            : adamw_by_count<P, G, MASTER, STATES_8_RANDOM>(a, wgs, s);
}
template <typename G>
hipError_t adamw_by_param(const AdamArgs& a, uint32_t wgs, int p_bf16, int mode, hipStream_t s) {
    if (!p_bf16) return adamw_by_mode<float, G, false>(a, wgs, mode, s);
    return a.master ? adamw_by_mode<bf16_t, G, true>(a, wgs, mode, s) : adamw_by_mode<bf16_t, G, false>(a, wgs, mode, s);
}

// Squares are summed in 64 bits: in 32 those of gradients above 2^64 or below
// 2^-75 would be lost. It costs no time: with fp32 products and sums 34 M bf16
// elements took as long (19.4 us against 19.6). The next vectors are loaded
// while these are summed.
template <typename G>
__device__ __forceinline__ double squares(const G* __restrict__ g, uint64_t n) {
    constexpr int N = 8, UV = 2;
    double sum[2] = {0., 0.};
    const uint64_t vecs = n / N;
    Vec<G, N> v[UV], next[UV];
    auto load = [&](Vec<G, N>(&q)[UV], uint64_t first) {
#pragma unroll
        for (int u = 0; u < UV; ++u) {
            q[u].zero();
            if (first + u * T < vecs) q[u].load(g + (first + u * T) * N);
        }
    };
    load(v, threadIdx.x);
    for (uint64_t first = threadIdx.x; first < vecs;) {
        first += UV * T;
        load(next, first);
#pragma unroll
        for (int u = 0; u < UV; ++u)
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const double x = v[u][k];
                sum[k % 2] = fma(x, x, sum[k % 2]);
            }
#pragma unroll
        for (int u = 0; u < UV; ++u) v[u] = next[u];
    }
    if (const uint64_t k = vecs * N + threadIdx.x; k < n) {
        const double x = widen(g[k]);
        sum[0] = fma(x, x, sum[0]);
    }
    return sum[0] + sum[1];
}

// Sum over a workgroup of N lanes in a fixed order, in lane 0.
template <int N>
__device__ __forceinline__ double wg_sum(double v) {
    __shared__ double part[N / 64];
#pragma unroll
    for (int d = 32; d >= 1; d /= 2) v += __shfl_xor(v, d);
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = v;
    __syncthreads();
    v = 0.;
    if (threadIdx.x == 0)
        for (int w = 0; w < N / 64; ++w) v += part[w];
    return v;
}

template <int TENSORS>
__global__ __launch_bounds__(T) void k_norm(NormTable<TENSORS> a) {
    const NormTensor& t = a.t[tensor_of(a, blockIdx.x)];
    const uint64_t address = (uint64_t)(t.w[1] & 0xffffu) << 32 | t.w[0],
                   count = ((uint64_t)(t.w[2] & 0x3ffffu) << 16 | t.w[1] >> 16) + 1,
                   at = (uint64_t)(blockIdx.x - first_wg(t)) * a.piece, n = min(a.piece, count - at);
    const double sum = wg_sum<T>(address & 1 ? squares((const bf16_t*)(address - 1) + at, n)
                                              : squares((const float*)address + at, n));
    if (threadIdx.x == 0) a.sums[blockIdx.x] = sum;
}

constexpr int TF = 1024;
// The sum is the first lane's.
__device__ __forceinline__ void norm_out(double sum, double max_norm, long long* step, float* out) {
    if (threadIdx.x > 0) return;
    const double norm = sqrt(sum);
    const bool finite = norm < (double)INFINITY;
    out[0] = (float)norm;
    out[1] = finite ? (float)fmin(1., max_norm / (norm + 1e-6)) : NAN;
    if (step && finite) ++*step;
}
__global__ __launch_bounds__(TF) void k_norm_finish(const double* sums, uint32_t n, double max_norm, long long* step,
                                                    float* out) {
    double sum = 0.;
    for (uint32_t i = threadIdx.x; i < n; i += 2 * TF) {   // both in flight: a launch leaves fewer than 2 TF
        const double a = sums[i], b = i + TF < n ? sums[i + TF] : 0.;
        sum += a + b;
    }
    norm_out(wg_sum<TF>(sum), max_norm, step, out);
}

// Few elements: one workgroup takes all pieces, each an entry of the table (no
// search), a wavefront one after the other, and finishes; the next entry is read
// while the present one's loads are in flight. One launch instead of two: a call
// takes 4.5 us instead of 6.9 for 10 x 2,000 fp32 elements, 5.8 instead of 6.8
// for 107,000; 131,072 are the same.
template <typename G>
__device__ __forceinline__ void add_piece(double (&sum)[2], const NormTensor& now, NormTensor& next, const NormTensor* after,
                                          uint32_t lane) {
    constexpr int N = 8, UV = NORM_PIECE / (64 * N);
    const G* g = (const G*)(((uint64_t)(now.w[1] & 0xffffu) << 32 | now.w[0]) & ~1ull);
    const uint32_t n = (now.w[1] >> 16) + 1;
    Vec<G, N> v[UV];
#pragma unroll
    for (int u = 0; u < UV; ++u) {
        const uint32_t at = (u * 64 + lane) * N;
        if (at + N <= n) {
            v[u].load(g + at);
        } else {
            v[u].zero();
            if (at < n) v[u].load_part(g + at, (int)(n - at));
        }
    }
    next = *after;
#pragma unroll
    for (int u = 0; u < UV; ++u)
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const double x = v[u][k];
            sum[k % 2] = fma(x, x, sum[k % 2]);
        }
}
__global__ __launch_bounds__(TF) void k_norm_alone(NormTable<NORM_PIECES> a, double max_norm, long long* step, float* out) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, n = (uint32_t)a.n;
    double sum[2] = {0., 0.};
    NormTensor next = a.t[wave];
    for (uint32_t p = wave; p < n;) {
        const NormTensor now = next;
        p += TF / 64;
        const NormTensor* after = &a.t[min(p, (uint32_t)NORM_PIECES - 1)];
        if (now.w[0] & 1)
            add_piece<bf16_t>(sum, now, next, after, lane);
        else
            add_piece<float>(sum, now, next, after, lane);
    }
    norm_out(wg_sum<TF>(sum[0] + sum[1]), max_norm, step, out);
}

}  // namespace

hipError_t adamw_launch(const AdamArgs& a, uint32_t wgs, int p_bf16, int g_bf16, int mode, hipStream_t s) {
    return g_bf16 ? adamw_by_param<bf16_t>(a, wgs, p_bf16, mode, s) : adamw_by_param<float>(a, wgs, p_bf16, mode, s);
}

hipError_t norm_launch(const NormArgs& a, uint32_t wgs, hipStream_t s) {
    if (a.n <= NORM_FEW)
        hipLaunchKernelGGL(k_norm<NORM_FEW>, dim3(wgs), dim3(T), 0, s, (shorter<NormHead, NormTable<NORM_FEW>>(a)));
    else
        hipLaunchKernelGGL(k_norm<NORM_TENSORS>, dim3(wgs), dim3(T), 0, s, a);
    return hipGetLastError();
}

hipError_t norm_alone(const NormTable<NORM_PIECES>& a, double max_norm, long long* step, float* out, hipStream_t s) {
    hipLaunchKernelGGL(k_norm_alone, dim3(1), dim3(TF), 0, s, a, max_norm, step, out);
    return hipGetLastError();
}

hipError_t norm_finish(const double* sums, uint32_t n, double max_norm, long long* step, float* out, hipStream_t s) {
    hipLaunchKernelGGL(k_norm_finish, dim3(1), dim3(TF), 0, s, sums, n, max_norm, step, out);
    return hipGetLastError();
}

}  // namespace wtc
