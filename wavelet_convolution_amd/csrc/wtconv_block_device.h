// Device-side helpers of the block operators: the counter generator, rows of
// eight channels, and reductions.
#pragma once

#include "wtconv_block.h"

namespace wtc {

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011): ten rounds of two 32 x 32 -> 64 bit products on a
// 128-bit counter, the key stepped by two constants each round.
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
    return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
}
struct Philox {
    uint32_t k0, k1, site, o0, o1;
    __device__ __forceinline__ Philox(const unsigned long long* rng, uint32_t site_) : site(site_) {
        const unsigned long long seed = rng[0], off = rng[1];
        // the same in every lane: scalar registers
        k0 = __builtin_amdgcn_readfirstlane((uint32_t)seed);
        k1 = __builtin_amdgcn_readfirstlane((uint32_t)(seed >> 32));
        o0 = __builtin_amdgcn_readfirstlane((uint32_t)off);
        o1 = __builtin_amdgcn_readfirstlane((uint32_t)(off >> 32));
    }
    __device__ __forceinline__ uint4 operator()(uint32_t group) const {
        uint32_t c0 = group, c1 = site, c2 = o0, c3 = o1, a = k0, b = k1;
        // the ten keys of each half are made again by the scalar unit, not
        // held in twenty of its registers
        asm volatile("" : "+s"(a), "+s"(b));
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            const uint64_t p = (uint64_t)c0 * 0xD2511F53u, q = (uint64_t)c2 * 0xCD9E8D57u;
            const uint32_t n0 = xor3((uint32_t)(q >> 32), c1, a), n2 = xor3((uint32_t)(p >> 32), c3, b);
            c1 = (uint32_t)q;
            c3 = (uint32_t)p;
            c0 = n0;
            c2 = n2;
            a += 0x9E3779B9u;
            b += 0xBB67AE85u;
        }
        return make_uint4(c0, c1, c2, c3);
    }
};

// Bit 7 - e set: element e of the group is dropped (the sign of its 16 bits
// less the threshold, shifted in from the right).
__device__ __forceinline__ uint32_t drop_bits(const uint4& r, uint32_t thr) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m = __builtin_amdgcn_alignbit(m, (w[i] & 0xffffu) - thr, 31);
        m = __builtin_amdgcn_alignbit(m, (w[i] >> 16) - thr, 31);
    }
    return m;
}
constexpr uint32_t ALL_DROPPED = 0xffu;

// v, or zero (whatever v is) where the bit is set: the bit spread over a
// word, without a comparison's lane mask.
__device__ __forceinline__ float zero_if(float v, uint32_t m, int bit) {
    const uint32_t d = (uint32_t)((int32_t)(m << (31 - bit)) >> 31);
    return __uint_as_float(__float_as_uint(v) & ~d);
}
__device__ __forceinline__ float kept(float v, uint32_t m, int e) { return zero_if(v, m, 7 - e); }

// Drop bits of the eight channels from c on, in a row whose first group is
// row_group: two generator groups where c is not a multiple of eight (the
// last lane of a row of an odd width).
__device__ __forceinline__ uint32_t drop_bits_at(const Philox& gen, uint32_t row_group, int c, bool odd, uint32_t thr) {
    const uint32_t g = row_group + (uint32_t)(c / CG);
    const uint32_t m = drop_bits(gen(g), thr);
    if (!odd) return m;   // the same for every lane
    const int s = c % CG;
    return s ? ((m << 8 | drop_bits(gen(g + 1), thr)) >> (8 - s)) & 0xffu : m;
}

// Whole samples take a counter of their own: the site with its top bit set.
__device__ __forceinline__ bool sample_kept(const BlockArgs& a, int b) {
    const Philox g(a.rng, a.site | 0x80000000u);
    return (g((uint32_t)b).x & 0xffffu) >= a.thr;
}

template <typename T> __device__ __forceinline__ T narrow_to(float f);
template <> __device__ __forceinline__ float narrow_to<float>(float f) { return f; }
template <> __device__ __forceinline__ bf16_t narrow_to<bf16_t>(float f) { return narrow_bf16(f); }

// Workgroups go to the eight XCDs in turn, each with an L2 of its own. The
// i-th of n workgroups takes this piece of work, so that neighbouring pieces
// (tiles of a plane that share a cache line) are on one XCD.
__device__ __forceinline__ unsigned xcd_order(unsigned i, unsigned n) {
    const unsigned xcd = i % 8, share = n / 8, more = n % 8;
    return xcd * share + min(xcd, more) + i / 8;
}

// Sum over aligned groups of N lanes (N a power of two up to 64), in every
// lane: data-parallel moves within a row of 16 lanes (pairs, quads, half
// mirror, mirror), then the two row swaps.
template <int CTRL>
__device__ __forceinline__ float dpp_mov(float v) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}
template <int N>
__device__ __forceinline__ float lane_sum(float v) {
    if constexpr (N >= 2) v += dpp_mov<0xB1>(v);    // lanes 1 0 3 2
    if constexpr (N >= 4) v += dpp_mov<0x4E>(v);    // lanes 2 3 0 1
    if constexpr (N >= 8) v += dpp_mov<0x141>(v);   // half mirror: the other quad of eight
    if constexpr (N >= 16) v += dpp_mov<0x140>(v);  // mirror: the other half of sixteen
    if constexpr (N >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if constexpr (N >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return v;
}
// v of lane K of each quad, in all four lanes.
template <int K>
__device__ __forceinline__ float quad_lane(float v) {
    return dpp_mov<K * 0x55>(v);   // lanes K K K K
}

// lane_sum over lanes N apart: lanes l, l + N, ... up to 64 (N >= 4).
template <int N>
__device__ __forceinline__ float stride_sum(float v) {
    if constexpr (N <= 4) v += dpp_mov<0x124>(v);   // rotate by 4 within sixteen,
    if constexpr (N <= 8) v += dpp_mov<0x128>(v);   // by 8
    if constexpr (N <= 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// N consecutive activations in their storage format, at addresses aligned to
// the element only (the vector memory unit takes 16 bytes at any such
// address). Where a row's or a plane's length is no multiple of the vector,
// its last vector moves back to end with it, and overlaps its neighbour.
typedef uint32_t words4 __attribute__((ext_vector_type(4)));
typedef uint32_t words2 __attribute__((ext_vector_type(2)));
typedef words4 words4_any __attribute__((aligned(2)));
typedef words2 words2_any __attribute__((aligned(2)));

template <typename T, int N>
struct Vec {
    static constexpr int WORDS = N * Act<T>::BYTES / 4;
    uint32_t w[WORDS];

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const T* __restrict__ p) {
        if constexpr (WORDS % 4 == 0) {
#pragma unroll
            for (int i = 0; i < WORDS; i += 4) {
                const words4 q = *(const words4_any*)((const char*)p + 4 * i);
                w[i] = q.x;
                w[i + 1] = q.y;
                w[i + 2] = q.z;
                w[i + 3] = q.w;
            }
        } else {
            static_assert(WORDS == 2, "");
            const words2 q = *(const words2_any*)p;
            w[0] = q.x;
            w[1] = q.y;
        }
    }
    // the first n elements, zeros past them
    __device__ __forceinline__ void load_part(const T* __restrict__ p, int n) {
        zero();
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) {
                if constexpr (sizeof(T) == 4)
                    w[i] = __float_as_uint(p[i]);
                else
                    w[i / 2] |= (uint32_t)p[i] << (16 * (i % 2));
            }
    }
    // as they are, without a rounding
    __device__ __forceinline__ void store(T* __restrict__ p) const {
        if constexpr (WORDS % 4 == 0) {
#pragma unroll
            for (int i = 0; i < WORDS; i += 4)
                *(words4_any*)((char*)p + 4 * i) = words4{w[i], w[i + 1], w[i + 2], w[i + 3]};
        } else {
            static_assert(WORDS == 2, "");
            *(words2_any*)p = words2{w[0], w[1]};
        }
    }
    __device__ __forceinline__ void store_part(T* __restrict__ p, int n) const {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) {
                if constexpr (sizeof(T) == 4)
                    p[i] = __uint_as_float(w[i]);
                else
                    p[i] = (T)(w[i / 2] >> (16 * (i % 2)));
            }
    }
    // zeros otherwise, whatever was loaded
    __device__ __forceinline__ void keep_if(bool yes) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = yes ? w[i] : 0u;
    }
    __device__ __forceinline__ void renew() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) asm volatile("" : "+v"(w[i]));
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        return __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
};

// N fp32 values, rounded to T.
template <typename T, int N>
__device__ __forceinline__ void store_vec(T* __restrict__ p, const float (&v)[N]) {
    constexpr int WORDS = N * Act<T>::BYTES / 4;
    uint32_t w[WORDS];
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
        if constexpr (sizeof(T) == 4)
            w[i] = __float_as_uint(v[i]);
        else
            w[i] = narrow_bf16x2(v[2 * i], v[2 * i + 1]);
    }
    if constexpr (WORDS % 4 == 0) {
#pragma unroll
        for (int i = 0; i < WORDS; i += 4) *(words4_any*)((char*)p + 4 * i) = words4{w[i], w[i + 1], w[i + 2], w[i + 3]};
    } else {
        static_assert(WORDS == 2, "");
        *(words2_any*)p = words2{w[0], w[1]};
    }
}
// The first n of them.
template <typename T, int N>
__device__ __forceinline__ void store_part(T* __restrict__ p, const float (&v)[N], int n) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < n) p[i] = narrow_to<T>(v[i]);
}

// Eight channels of a parameter from c on; `none` where there is no such
// parameter. PART: the first n channels only.
template <bool PART = false>
__device__ __forceinline__ void load_param_if(bool has, const float* __restrict__ p, int c, float none, float (&v)[CG],
                                              int n = CG) {
    if (!has) {
#pragma unroll
        for (int i = 0; i < CG; ++i) v[i] = none;
        return;
    }
    // loaded where it is used: held over a loop, parameters cost more
    // registers than their next read from cache costs time
    asm volatile("" : "+v"(c));
    Vec<float, CG> q;
    if constexpr (PART)
        q.load_part(p, n);
    else
        q.load(p + c);
#pragma unroll
    for (int i = 0; i < CG; ++i) v[i] = q[i];
}
template <bool PART = false>
__device__ __forceinline__ void load_param(const float* __restrict__ p, int c, float none, float (&v)[CG], int n = CG) {
    load_param_if<PART>(p != nullptr, p, c, none, v, n);
}

// Eight channels by PV pixels in a lane's registers, from either memory order.
template <typename T, bool CLAST, int PV>
struct Patch {   // [8 channels] x [PV pixels]
    static constexpr int NVEC = CLAST ? PV : CG, LEN = CLAST ? CG : PV;
    Vec<T, LEN> v[NVEC];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < NVEC; ++i) v[i].zero();
    }
    // p is the sample's first element, the same for every lane, and off
    // (bytes) the lane's place in it
    __device__ __forceinline__ void load(const T* __restrict__ p, uint32_t off, size_t step) {
#pragma unroll
        for (int i = 0; i < NVEC; ++i) v[i].load((const T*)((const char*)(p + i * step) + off));
    }
    // From here on the words are new to the compiler: what it made of them
    // before (widened values, twice the registers in bf16) is made again
    // rather than held.
    __device__ __forceinline__ void renew() {
#pragma unroll
        for (int i = 0; i < NVEC; ++i) v[i].renew();
    }
    // zeros in the place of what is dropped
    template <class D>
    __device__ __forceinline__ void drop(const D& m) {
        constexpr int PER = 4 / (int)sizeof(T);   // elements a word
#pragma unroll
        for (int i = 0; i < NVEC; ++i)
#pragma unroll
            for (int k = 0; k < LEN; k += PER) {
                const uint32_t lo = CLAST ? m.spread(k, i) : m.spread(i, k);
                uint32_t gone = lo;
                if constexpr (PER == 2) {
                    const uint32_t hi = CLAST ? m.spread(k + 1, i) : m.spread(i, k + 1);
                    gone = (lo & 0xffffu) | (hi & 0xffff0000u);
                }
                v[i].w[k / PER] &= ~gone;
            }
    }
    __device__ __forceinline__ float at(int ch, int px) const { return CLAST ? v[px][ch] : v[ch][px]; }
};

// f(channel, pixel) for every element, rounded and stored.
template <typename T, bool CLAST, int PV, class F>
__device__ __forceinline__ void store_patch(T* __restrict__ p, uint32_t off, size_t step, F&& f) {
    constexpr int NVEC = CLAST ? PV : CG, LEN = CLAST ? CG : PV;
#pragma unroll
    for (int i = 0; i < NVEC; ++i) {
        float o[LEN];
#pragma unroll
        for (int k = 0; k < LEN; ++k) o[k] = CLAST ? f(k, i) : f(i, k);
        store_vec<T, LEN>((T*)((char*)(p + i * step) + off), o);
        __builtin_amdgcn_sched_barrier(0);   // a vector at a time: fewer values in flight
    }
}

// Drop bits of a lane's elements: a byte for each pixel, the first at the top
// of a word.
template <int PV>
struct Drops {
    static_assert(PV % 4 == 0, "");
    uint32_t w[PV / 4];
    template <bool ODD>
    __device__ __forceinline__ void draw(const BlockArgs& a, uint32_t row, int c) {
        const Philox gen(a.rng, a.site);
        const uint32_t G = (uint32_t)cdiv(a.C, CG);
        uint32_t g = row * G;   // fewer than 2^32 groups in all
#pragma unroll
        for (int k = 0; k < PV / 4; ++k) {
            uint32_t m = 0;
#pragma unroll 2
            for (int j = 0; j < 4; ++j, g += G) m = m << 8 | drop_bits_at(gen, g, c, ODD, a.thr);
            w[k] = m;
        }
    }
    __device__ __forceinline__ float kept(float v, int i, int j) const {
        return zero_if(v, w[j / 4], bit(i, j));
    }
    // all ones where the element is dropped
    __device__ __forceinline__ uint32_t spread(int i, int j) const {
        return (uint32_t)((int32_t)(w[j / 4] << (31 - bit(i, j))) >> 31);
    }
    static constexpr int bit(int i, int j) { return 8 * (3 - j % 4) + 7 - i; }
};

}  // namespace wtc
