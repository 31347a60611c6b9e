// Slots sorted by expert (a stable counting sort). A wavefront owns a run of
// consecutive slots: it counts them by expert in LDS, the counts of all
// wavefronts before it give each expert's first place, and it walks its run
// once more, 64 slots at a time; slots of one expert among the 64 are found
// by a ballot over each bit of the expert's number, so that a slot's rank is
// a population count and no atomic decides an order.
#include "wtconv_experts.h"

namespace wtc {
namespace {

constexpr int T = 1024, WAVES = T / 64;

// One workgroup sorts this many slots by itself; more of them are cut into
// parts, whose counts a first launch leaves in the workspace.
constexpr uint32_t ALONE = 8192;

// The slot's expert; E where it has none.
template <typename I>
__device__ __forceinline__ int key_of(const SortArgs& a, uint32_t slot) {
    const I e = ((const I*)a.expert)[slot];
    return e >= 0 && e < (I)a.E ? (int)e : a.E;
}

// f(first slot of 64, how many) over wavefront w's run of the slots
// [begin, end): whole groups of 64, each a wavefront's at once.
template <class F>
__device__ __forceinline__ void each_group(uint32_t begin, uint32_t end, int w, F&& f) {
    const uint32_t groups = (end - begin + 63) / 64, per = (groups + WAVES - 1) / WAVES;
    const uint32_t first = min(groups, w * per), last = min(groups, first + per);
    for (uint32_t g = first; g < last; ++g) f(begin + g * 64, min(64u, end - begin - g * 64));
}

// cnt[w][e]: the slots of expert e in wavefront w's run.
template <typename I>
__device__ __forceinline__ void count_runs(const SortArgs& a, uint32_t begin, uint32_t end, int* cnt) {
    const int n = a.E + 1, w = threadIdx.x / 64, lane = threadIdx.x % 64;
    for (int i = threadIdx.x; i < WAVES * n; i += T) cnt[i] = 0;
    __syncthreads();
    each_group(begin, end, w, [&](uint32_t at, uint32_t len) {
        if ((uint32_t)lane < len) atomicAdd(&cnt[w * n + key_of<I>(a, at + lane)], 1);   // counts: any order
    });
    __syncthreads();
}

template <typename I>
__global__ __launch_bounds__(T) void k_sort_count(SortArgs a) {
    __shared__ int cnt[WAVES * (MAX_EXPERTS + 1)];
    const uint32_t begin = min(a.S, blockIdx.x * a.per);   // the last parts may be empty
    count_runs<I>(a, begin, min(a.S, begin + a.per), cnt);
    const int n = a.E + 1;
    for (int e = threadIdx.x; e < n; e += T) {
        int sum = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) sum += cnt[w * n + e];
        a.counts[(size_t)blockIdx.x * n + e] = sum;
    }
}

template <typename I>
__global__ __launch_bounds__(T) void k_sort_place(SortArgs a) {
    __shared__ int cnt[WAVES * (MAX_EXPERTS + 1)];
    __shared__ int all[MAX_EXPERTS + 1], before[MAX_EXPERTS + 1];   // of all parts; of those before this one
    const int n = a.E + 1, w = threadIdx.x / 64, lane = threadIdx.x % 64;
    const uint32_t part = blockIdx.x, begin = min(a.S, part * a.per), end = min(a.S, begin + a.per);
    for (int e = threadIdx.x; e < n; e += T) all[e] = before[e] = 0;
    count_runs<I>(a, begin, end, cnt);   // with barriers
    if (a.parts == 1) {
        for (int e = threadIdx.x; e < n; e += T) {
            int sum = 0;
#pragma unroll
            for (int k = 0; k < WAVES; ++k) sum += cnt[k * n + e];
            all[e] = sum;
        }
    } else {
        // a thread sums one expert's counts of every `slices`-th part
        const int wide = n > T / 2 ? T : 1 << (32 - __clz(n - 1)), slices = T / wide;
        for (int e = threadIdx.x % wide; e < n; e += wide) {
            int sum = 0, mine = 0;
#pragma unroll 8
            for (int p = threadIdx.x / wide; p < a.parts; p += slices) {
                const int c = a.counts[(size_t)p * n + e];
                sum += c;
                mine += p < (int)part ? c : 0;
            }
            if (slices == 1) {
                all[e] = sum;
                before[e] = mine;
            } else {   // whole numbers: any order
                atomicAdd(&all[e], sum);
                atomicAdd(&before[e], mine);
            }
        }
    }
    __syncthreads();
    // each expert's first place: the sums before it, 64 runs of experts in a
    // wavefront's lanes
    if (w == 0) {
        const int per = (n + 63) / 64, first = min(n, lane * per), last = min(n, first + per);
        int sum = 0;
        for (int e = first; e < last; ++e) sum += all[e];
        int up = sum;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(up, d);
            up += lane >= d ? o : 0;
        }
        int at = up - sum;
        for (int e = first; e < last; ++e) {
            const int c = all[e];
            all[e] = at;
            at += c;
        }
    }
    __syncthreads();
    // each wavefront's first place of each expert
    for (int e = threadIdx.x; e < n; e += T) {
        if (part == 0) a.offsets[e] = all[e];
        int at = all[e] + before[e];
#pragma unroll
        for (int k = 0; k < WAVES; ++k) {
            const int c = cnt[k * n + e];
            cnt[k * n + e] = at;
            at += c;
        }
    }
    __syncthreads();
    const int bits = 32 - __clz(a.E);   // of the numbers 0..E
    each_group(begin, end, w, [&](uint32_t at, uint32_t len) {
        const bool on = (uint32_t)lane < len;
        const int e = on ? key_of<I>(a, at + lane) : 0;
        uint64_t same = __ballot(on);
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot(e >> b & 1);
            same &= e >> b & 1 ? set : ~set;
        }
        const int rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32),
                                                   __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0));
        if (on) {
            const int first = cnt[w * n + e], p = first + rank;
            a.place[at + lane] = p;
            a.order[p] = (int)(at + lane);
            // one lane of each expert moves its count on, after all have read
            // it: a wavefront's LDS accesses are in order
            if (rank == 0) cnt[w * n + e] = first + (int)__popcll(same);
        }
        // the next group's reads stay behind this one's writes
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    });
}

// Slots go to as many workgroups as leave each 2,048 of them (two groups a
// wavefront), but to fewer where many experts would make the counts that
// every workgroup reads long.
int parts_of(long long S, int E) {
    if (S <= ALONE) return 1;
    long long most = 65536 / (E + 1);
    most = most < 32 ? 32 : most > 256 ? 256 : most;
    const long long p = (S + 2047) / 2048;
    return (int)(p < most ? p : most);
}

}  // namespace

size_t expert_sort_bytes(long long S, int E) {
    const int parts = parts_of(S, E);
    return parts == 1 ? 0 : (size_t)parts * (E + 1) * sizeof(int);
}

hipError_t expert_sort(SortArgs a, int id64, hipStream_t s) {
    a.parts = parts_of(a.S, a.E);
    a.per = (uint32_t)(((long long)a.S + a.parts - 1) / a.parts);
    a.per = (a.per + 63) / 64 * 64;
    if (a.parts > 1) {
        if (id64)
            hipLaunchKernelGGL(k_sort_count<int64_t>, dim3(a.parts), dim3(T), 0, s, a);
        else
            hipLaunchKernelGGL(k_sort_count<int32_t>, dim3(a.parts), dim3(T), 0, s, a);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    if (id64)
        hipLaunchKernelGGL(k_sort_place<int64_t>, dim3(a.parts), dim3(T), 0, s, a);
    else
        hipLaunchKernelGGL(k_sort_place<int32_t>, dim3(a.parts), dim3(T), 0, s, a);
    return hipGetLastError();
}

}  // namespace wtc
