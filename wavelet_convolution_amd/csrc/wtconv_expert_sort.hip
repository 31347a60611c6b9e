// Slots sorted by expert (a stable counting sort). A wavefront owns a run of
// consecutive slots: it counts them by expert in LDS, the counts of all
// wavefronts before it give each expert's first place, and it walks its run
// once more, 64 slots at a time; slots of one expert among the 64 are found
// by a ballot over each bit of the expert's number, so that a slot's rank is
// a population count and no atomic decides an order.
//
// What bounds it is the length of that chain, not memory: one workgroup sorts
// few slots alone (SORT_ALONE); else a first launch counts parts of some thousand
// slots and each part's workgroup sums up the counts of all (SORT_SUMS), or, where
// those are many, a launch in between makes running sums of them (SORT_SCAN).
// 16 experts: 2 slots 3.3 us, 4,096 5.5, 401,408 9.9 us (their 6.4 MB take 1.2);
// 64 experts: 8.4 M slots 74 us, 1.8 TB/s.
#include <algorithm>

#include "wtconv_experts.h"

namespace wtc {
namespace {

constexpr int T = 1024, WAVES = T / 64;

// Groups of 64 slots whose experts a wavefront holds in registers from its
// count to its walk; runs of more read them again.
constexpr int HELD = 4;
constexpr uint32_t MOST_HELD = WAVES * 64 * HELD;   // slots of a workgroup that are all held

enum { SORT_ALONE = 0, SORT_SUMS = 1, SORT_SCAN = 2 };

// The slot's expert; E where it has none.
template <typename I>
__device__ __forceinline__ int key_of(const SortArgs& a, uint32_t slot) {
    const I e = ((const I*)a.expert)[slot];
    return e >= 0 && e < (I)a.E ? (int)e : a.E;
}

// Wavefront w's run of the slots [begin, end): groups of 64, the last one of
// all perhaps of fewer.
struct Run {
    uint32_t first, last, end;   // slots: of the first group, past the last group, past the last slot
    int waves;                   // wavefronts that have a group
    __device__ __forceinline__ Run(uint32_t begin, uint32_t stop, uint32_t w) : end(stop) {
        const uint32_t groups = (stop - begin + 63) / 64, per = (groups + WAVES - 1) / WAVES;
        first = begin + min(groups, w * per) * 64;
        last = begin + min(groups, w * per + per) * 64;
        waves = per ? (int)((groups + per - 1) / per) : 0;
    }
};

// The experts of a run, a group after the other: held, or read at each use.
template <typename I, bool ALL>
struct Keys {
    int held[ALL ? HELD : 1];
    __device__ __forceinline__ void load(const SortArgs& a, const Run& r, uint32_t lane) {
        if constexpr (ALL) {
#pragma unroll
            for (int g = 0; g < HELD; ++g) {
                const uint32_t slot = r.first + g * 64 + lane;
                held[g] = r.first + g * 64 < r.last && slot < r.end ? key_of<I>(a, slot) : -1;
            }
        }
    }
    // f(first slot of the group, this lane's expert, or -1 past the end)
    template <class F>
    __device__ __forceinline__ void each(const SortArgs& a, const Run& r, uint32_t lane, F&& f) const {
        if constexpr (ALL) {
#pragma unroll
            for (int g = 0; g < HELD; ++g)
                if (r.first + g * 64 < r.last) f(r.first + g * 64, held[g]);
        } else {
            for (uint32_t at = r.first; at < r.last; at += 64)
                f(at, at + lane < r.end ? key_of<I>(a, at + lane) : -1);
        }
    }
};

// By parts, or by experts where k_sort_scan goes over an expert's parts.
template <typename I>
__global__ __launch_bounds__(T) void k_sort_count(SortArgs a, bool by_expert) {
    __shared__ int cnt[MAX_EXPERTS + 1];
    const uint32_t w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const uint32_t begin = min(a.S, blockIdx.x * a.per), end = min(a.S, begin + a.per);   // the last parts may be empty
    const int n = a.E + 1;
    for (int e = threadIdx.x; e < n; e += T) cnt[e] = 0;
    __syncthreads();
    Keys<I, false>().each(a, Run(begin, end, w), lane, [&](uint32_t, int e) {
        if (e >= 0) atomicAdd(&cnt[e], 1);   // counts: any order
    });
    __syncthreads();
    for (int e = threadIdx.x; e < n; e += T)
        a.counts[by_expert ? (size_t)e * a.parts + blockIdx.x : (size_t)blockIdx.x * n + e] = cnt[e];
}

__device__ __forceinline__ int wave_before(int v, int lane) {   // of the lanes before
    int up = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(up, d);
        up += lane >= d ? o : 0;
    }
    return up - v;
}

// Running sums of one expert's counts over the parts, in their place, and their
// total behind all counts: a workgroup an expert.
__global__ __launch_bounds__(T) void k_sort_scan(SortArgs a) {
    __shared__ int of[WAVES];
    const int w = threadIdx.x / 64, lane = threadIdx.x % 64, n = a.E + 1;
    int* counts = a.counts + (size_t)blockIdx.x * a.parts;
    int done = 0;
    for (int p0 = 0; p0 < a.parts; p0 += T) {
        const int p = p0 + (int)threadIdx.x, c = p < a.parts ? counts[p] : 0, before = wave_before(c, lane);
        if (lane == 63) of[w] = before + c;
        __syncthreads();
        int at = done;
#pragma unroll
        for (int k = 0; k < WAVES; ++k) {
            at += k < w ? of[k] : 0;
            done += of[k];
        }
        if (p < a.parts) counts[p] = at + before;
        __syncthreads();
    }
    if (threadIdx.x == 0) a.counts[(size_t)n * a.parts + blockIdx.x] = done;
}

template <typename I, bool ALL, int MODE>
__global__ __launch_bounds__(T) void k_sort_place(SortArgs a) {
    __shared__ int cnt[WAVES * (MAX_EXPERTS + 1)];                  // a wavefront's slots of an expert; then its next place
    __shared__ int all[MAX_EXPERTS + 1], before[MAX_EXPERTS + 1];   // of all parts; of those before this one
    const uint32_t w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const int n = a.E + 1;
    const uint32_t part = blockIdx.x, begin = min(a.S, part * a.per), end = min(a.S, begin + a.per);
    const Run run(begin, end, w);
    Keys<I, ALL> keys;
    keys.load(a, run, lane);
    // a thread sums up one expert's counts in every `slices`-th part
    const int wide = n > T / 2 ? T : 1 << (32 - __clz(n - 1)), mine = threadIdx.x % wide;
    int sum[2] = {0, 0}, less[2] = {0, 0};   // two experts where there is one more than threads
    if constexpr (MODE == SORT_SUMS) {
#pragma unroll 8
        for (int p = threadIdx.x / wide; p < a.parts; p += T / wide) {
            const int c = mine < n ? a.counts[(size_t)p * n + mine] : 0;
            sum[0] += c;
            less[0] += p < (int)part ? c : 0;
        }
        if (mine + T < n)
            for (int p = 0; p < a.parts; ++p) {
                const int c = a.counts[(size_t)p * n + mine + T];
                sum[1] += c;
                less[1] += p < (int)part ? c : 0;
            }
        for (int e = threadIdx.x; e < n; e += T) all[e] = before[e] = 0;
    }
    if constexpr (MODE == SORT_SCAN) {
        for (int e = threadIdx.x; e < n; e += T) {
            all[e] = a.counts[(size_t)n * a.parts + e];
            before[e] = a.counts[(size_t)e * a.parts + part];
        }
    }
    for (int i = threadIdx.x; i < run.waves * n; i += T) cnt[i] = 0;
    __syncthreads();
    keys.each(a, run, lane, [&](uint32_t, int e) {
        if (e >= 0) atomicAdd(&cnt[w * n + e], 1);   // counts, here and below: any order
    });
    if constexpr (MODE == SORT_SUMS) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (const int e = mine + i * T; e < n) {
                atomicAdd(&all[e], sum[i]);
                atomicAdd(&before[e], less[i]);
            }
    }
    __syncthreads();
    int* next = cnt + w * n;   // of each expert, the wavefront's next place
    if (MODE == SORT_ALONE && n <= 64) {
        // every wavefront for itself, an expert a lane, without the three barriers
        // below: 256 slots of 16 experts 3.4 us against 4.0, 4,096 5.5 against 5.9;
        // more experts, and parts' workgroups, were slower
        next += WAVES * n;
        const int e = min((int)lane, n - 1);
        int of_before = 0, of_all = 0;   // of the wavefronts
        for (int k = 0; k < run.waves; ++k) {
            const int c = cnt[k * n + e];
            of_before += k < (int)w ? c : 0;
            of_all += c;
        }
        const int first = wave_before((int)lane < n ? of_all : 0, (int)lane);
        if ((int)lane < n) {
            if (w == 0) a.offsets[e] = first;
            next[e] = first + of_before;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    } else {
        if constexpr (MODE == SORT_ALONE) {
            for (int e = threadIdx.x; e < n; e += T) {
                int c = 0;
                for (int k = 0; k < run.waves; ++k) c += cnt[k * n + e];
                all[e] = c;
                before[e] = 0;
            }
            __syncthreads();
        }
        // each expert's first place: the sums before it, 64 runs of experts in a
        // wavefront's lanes
        if (w == 0) {
            const int per = (n + 63) / 64, first = min(n, (int)lane * per), last = min(n, first + per);
            int c = 0;
            for (int e = first; e < last; ++e) c += all[e];
            int at = wave_before(c, (int)lane);
            for (int e = first; e < last; ++e) {
                const int here = all[e];
                all[e] = at;
                at += here;
            }
        }
        __syncthreads();
        // each wavefront's first place of each expert
        for (int e = threadIdx.x; e < n; e += T) {
            if (part == 0) a.offsets[e] = all[e];
            int at = all[e] + before[e];
            for (int k = 0; k < run.waves; ++k) {
                const int c = cnt[k * n + e];
                cnt[k * n + e] = at;
                at += c;
            }
        }
        __syncthreads();
    }
    const int bits = 32 - __clz(a.E);   // of the numbers 0..E
    keys.each(a, run, lane, [&](uint32_t at, int e) {
        const bool on = e >= 0;
        // lanes whose expert agrees in every bit: as all ones or none a bit costs
        // five instructions (4,096 slots of 64 experts 6.1 us; 6.7 with a choice
        // between two masks, at eleven)
        const uint64_t all_on = __ballot(on);
        uint32_t lo = (uint32_t)all_on, hi = (uint32_t)(all_on >> 32);
        for (int left = 31; left > 31 - bits; --left) {
            const uint32_t bit = (uint32_t)((int)((uint32_t)e << left) >> 31);
            const uint64_t set = __ballot(bit != 0);
            lo &= ~((uint32_t)set ^ bit);
            hi &= ~((uint32_t)(set >> 32) ^ bit);
        }
        const int rank = __builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0));
        if (on) {
            const int first = next[e], p = first + rank;
            // one lane of each expert moves its count on, after all have read
            // it: a wavefront's LDS accesses are in order, and the compiler
            // keeps the reads before the fence
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            a.place[at + lane] = p;
            a.order[p] = (int)(at + lane);
            if (rank == 0) next[e] = first + __popc(lo) + __popc(hi);
        }
        // the next group's reads stay behind this one's writes
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    });
}

// How S slots of E experts are sorted, in how many parts. Alone up to what the
// wavefronts of a workgroup hold: 4,096 slots of 64 experts 6.1 us against 6.9
// in parts, 8,192 in two rounds 10.7 against 7.4.
struct Plan {
    int mode, parts;
    uint32_t per;
};
// Parts of 2,048 slots; of 1,024 where a part's workgroup has few counts to sum
// up and a CU to itself (65,536 slots of 64 experts 7.8 us against 8.9, of 128
// experts 8.8 against 8.7), and of 4,096 where the card would not hold all of
// 2,048 at once (2.1 M slots of 16 experts 17.4 against 22, 1.05 M the same).
// The sums cost every part's workgroup the counts of all parts, in rows of a power
// of two, and the running sums a launch: 401,408 slots of 64 experts (196 rows of
// 128) 11.1 us against 11.7, 262,144 of 128 (128 of 256) 11.5 and 11.7, 300,000 of
// 128 12.8 and 12.0; with two workgroups a CU 600,000 of 32 (293 of 64) 12.2 and
// 12.4, of 64 16.2 and 13.3. The number of parts is bounded, so beyond 2^24 slots
// a part has more than its wavefronts hold: those are for the kernel that reads
// experts again, which goes by running sums (2^24 + 1 slots of 3 experts 114 us,
// 2^24 of them 126 by sums).
Plan plan_of(long long S, int E) {
    constexpr long long MOST = 4096;
    if (S <= MOST_HELD) return {SORT_ALONE, 1, (uint32_t)S};
    long long row = 2;
    while (row < E + 1) row *= 2;
    auto count = [&](long long part) { return std::min((S + part - 1) / part, MOST); };
    const long long parts = count(S > 512 * 2048 ? 4096 : S <= 256 * 1024 && count(1024) * row <= 12288 ? 1024 : 2048);
    const long long per = ((S + parts - 1) / parts + 63) / 64 * 64;   // the last parts may be short or empty
    const bool sums = per <= MOST_HELD && parts * row <= (parts <= 256 ? 32768 : 20480);
    return {sums ? SORT_SUMS : SORT_SCAN, (int)parts, (uint32_t)per};
}

template <typename I, bool ALL>
void place(const SortArgs& a, int mode, hipStream_t s) {
    if (mode == SORT_ALONE)
        hipLaunchKernelGGL((k_sort_place<I, true, SORT_ALONE>), dim3(1), dim3(T), 0, s, a);
    else if (mode == SORT_SUMS)
        hipLaunchKernelGGL((k_sort_place<I, true, SORT_SUMS>), dim3(a.parts), dim3(T), 0, s, a);
    else
        hipLaunchKernelGGL((k_sort_place<I, ALL, SORT_SCAN>), dim3(a.parts), dim3(T), 0, s, a);
}

template <typename I>
hipError_t sort(const SortArgs& a, int mode, hipStream_t s) {
    // held slots past the last group would be neither counted nor placed
    const bool held = a.per <= MOST_HELD;
    if (!held && mode != SORT_SCAN) return hipErrorInvalidConfiguration;
    if (mode != SORT_ALONE) {
        hipLaunchKernelGGL(k_sort_count<I>, dim3(a.parts), dim3(T), 0, s, a, mode == SORT_SCAN);
        if (mode == SORT_SCAN) hipLaunchKernelGGL(k_sort_scan, dim3(a.E + 1), dim3(T), 0, s, a);
    }
    if (held)
        place<I, true>(a, mode, s);
    else
        place<I, false>(a, mode, s);
    return hipGetLastError();
}

}  // namespace

size_t expert_sort_bytes(long long S, int E) {
    const Plan p = plan_of(S, E);
    return p.mode == SORT_ALONE ? 0 : (size_t)(p.parts + 1) * (E + 1) * sizeof(int);
}

hipError_t expert_sort(SortArgs a, int id64, hipStream_t s) {
    const Plan p = plan_of(a.S, a.E);
    a.parts = p.parts;
    a.per = p.per;
    return id64 ? sort<int64_t>(a, p.mode, s) : sort<int32_t>(a, p.mode, s);
}

}  // namespace wtc
