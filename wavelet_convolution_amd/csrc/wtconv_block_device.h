// Device-side helpers of the block operators: the counter generator, rows of
// eight channels, and reductions.
#pragma once

#include "wtconv_block.h"

namespace wtc {

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011): ten rounds of two 32 x 32 -> 64 bit products on a
// 128-bit counter, the key stepped by two constants each round.
struct Philox {
    uint32_t k0, k1, site, o0, o1;
    __device__ __forceinline__ Philox(const unsigned long long* rng, uint32_t site_) : site(site_) {
        const unsigned long long seed = rng[0], off = rng[1];
        k0 = (uint32_t)seed;
        k1 = (uint32_t)(seed >> 32);
        o0 = (uint32_t)off;
        o1 = (uint32_t)(off >> 32);
    }
    __device__ __forceinline__ uint4 operator()(uint32_t group) const {
        uint32_t c0 = group, c1 = site, c2 = o0, c3 = o1, a = k0, b = k1;
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            const uint64_t p = (uint64_t)c0 * 0xD2511F53u, q = (uint64_t)c2 * 0xCD9E8D57u;
            const uint32_t n0 = (uint32_t)(q >> 32) ^ c1 ^ a, n2 = (uint32_t)(p >> 32) ^ c3 ^ b;
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

// Bit e set: element e of the group is kept.
__device__ __forceinline__ uint32_t keep_bits(const uint4& r, uint32_t thr) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m |= ((w[i] & 0xffffu) >= thr ? 1u : 0u) << (2 * i);
        m |= ((w[i] >> 16) >= thr ? 1u : 0u) << (2 * i + 1);
    }
    return m;
}

// Whole samples take a counter of their own: the site with its top bit set.
__device__ __forceinline__ bool sample_kept(const BlockArgs& a, int b) {
    const Philox g(a.rng, a.site | 0x80000000u);
    return (g((uint32_t)b).x & 0xffffu) >= a.thr;
}

template <typename T> __device__ __forceinline__ T narrow_to(float f);
template <> __device__ __forceinline__ float narrow_to<float>(float f) { return f; }
template <> __device__ __forceinline__ bf16_t narrow_to<bf16_t>(float f) { return narrow_bf16(f); }

}  // namespace wtc
