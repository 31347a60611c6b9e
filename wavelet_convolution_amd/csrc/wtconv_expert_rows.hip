// Rows to their experts and back. Every kernel goes by rows n: what a row has
// in [N][C] is read or written once, and its K rows among the sorted ones are
// reached through place[n][k] (4 bytes a slot against 2 C), whichever side is
// read. Memory is the bound in each (bf16, copy rate of the card 5.2 TB/s):
// 401,408 slots of 96 channels there 20.3 us, 5.7 TB/s, weighted sum 23.2, 5.1,
// its gradient 42.0, 4.6; 100,352 of 768 channels 38.5, 40.7 and 78.1 us, 5.9,
// 5.7 and 4.9 TB/s.
#include "wtconv_block_device.h"
#include "wtconv_experts.h"

namespace wtc {
namespace {

constexpr int T = 256;

// A slot's row among the sorted ones: whether there is one (a place that is no
// place would be out of bounds), and whether it belongs to an expert.
struct Slot {
    uint32_t at;
    bool is, live;
};
__device__ __forceinline__ Slot slot_of(uint32_t at, uint32_t S, uint32_t kept) {
    return {at, at < S, at < S && at < kept};
}
__device__ __forceinline__ uint32_t kept_of(const ExpertArgs& a) {
    const int n = a.offsets[a.E];
    return n > 0 ? (uint32_t)n : 0u;
}

// A thread takes eight channels of a row (one vector; where C is no multiple
// of eight the last one moves back to end with the row and stores its
// neighbour's values once more), and KK slots at a time, whose reads are in
// flight together. More vectors a thread were slower: 401,408 slots of 96 bf16
// channels, weighted sum 23.1 us, 24.2 with two and 26.7 with four.
template <typename X, int OP, int KK, bool PART>
__global__ __launch_bounds__(T) void k_expert_move(ExpertArgs a, uint32_t G, uint64_t wgs) {
    const uint32_t S = (uint32_t)(a.N * a.K), kept = kept_of(a);
    for (uint64_t wg = blockIdx.x; wg < wgs; wg += gridDim.x) {
        const uint64_t first = wg * T, row0 = first / G;   // scalar
        const uint32_t t = (uint32_t)(first - row0 * G) + threadIdx.x, down = t / G;
        const uint64_t row = row0 + down;
        if (row >= (uint64_t)a.N) return;
        const uint32_t c = PART ? 0 : min((t - down * G) * CG, (uint32_t)a.C - CG);
        auto load = [&](Vec<X, CG>& v, const void* rows, uint64_t at) {
            const X* p = (const X*)rows + at * a.C;
            if constexpr (PART)
                v.load_part(p, a.C);
            else
                v.load(p + c);
        };
        Vec<X, CG> x;
        float sum[CG] = {};
        if constexpr (OP == ROWS_FWD) load(x, a.rows, row);
        for (int k = 0; k < a.K; k += KK) {
            Slot s[KK];
            float w[KK];
#pragma unroll
            for (int i = 0; i < KK; ++i) {
                const bool is = k + i < a.K;
                s[i] = slot_of(is ? (uint32_t)a.place[row * a.K + k + i] : ~0u, S, kept);
                if constexpr (OP == SUM_FWD) w[i] = is ? a.w[row * a.K + k + i] : 0.f;
            }
            if constexpr (OP == ROWS_FWD) {
#pragma unroll
                for (int i = 0; i < KK; ++i) {
                    if (!s[i].is) continue;
                    Vec<X, CG> o = x;
                    if (!s[i].live) o.zero();
                    X* p = (X*)a.to_sorted + (size_t)s[i].at * a.C;
                    if constexpr (PART)
                        o.store_part(p, a.C);
                    else
                        o.store(p + c);
                }
            } else {
                Vec<X, CG> q[KK];
#pragma unroll
                for (int i = 0; i < KK; ++i) {
                    load(q[i], a.sorted, s[i].live ? s[i].at : 0);
                    q[i].keep_if(s[i].live);
                }
#pragma unroll
                for (int i = 0; i < KK; ++i) {
                    const float f = OP == ROWS_BWD ? 1.f : s[i].live ? w[i] : 0.f;
#pragma unroll
                    for (int j = 0; j < CG; ++j) sum[j] = fmaf(f, q[i][j], sum[j]);
                }
            }
        }
        if constexpr (OP != ROWS_FWD) {
            X* p = (X*)a.to_rows + row * a.C;
            if constexpr (PART)
                store_part<X, CG>(p, sum, a.C);
            else
                store_vec<X, CG>(p + c, sum);
        }
    }
}

// A grid of at most 2^31 lanes takes any number of pieces.
unsigned grid_of(uint64_t wgs) { return (unsigned)(wgs < 1u << 23 ? wgs : 1u << 23); }

template <typename X, int OP, int KK>
hipError_t move_launch(const ExpertArgs& a, hipStream_t s) {
    const uint32_t G = (uint32_t)cdiv(a.C, CG);
    const uint64_t wgs = ((uint64_t)a.N * G + T - 1) / T;
    if (a.C < CG)
        hipLaunchKernelGGL((k_expert_move<X, OP, KK, true>), dim3(grid_of(wgs)), dim3(T), 0, s, a, G, wgs);
    else
        hipLaunchKernelGGL((k_expert_move<X, OP, KK, false>), dim3(grid_of(wgs)), dim3(T), 0, s, a, G, wgs);
    return hipGetLastError();
}

// Slots at a time: see sum_bwd_by_k.
template <typename X, int OP>
hipError_t move_by_k(const ExpertArgs& a, hipStream_t s) {
    if (a.K == 1) return move_launch<X, OP, 1>(a, s);
    if (a.K == 2) return move_launch<X, OP, 2>(a, s);
    return move_launch<X, OP, 4>(a, s);
}

template <typename X>
hipError_t move_by_op(const ExpertArgs& a, int op, hipStream_t s) {
    if (op == ROWS_FWD) return move_by_k<X, ROWS_FWD>(a, s);
    if (op == ROWS_BWD) return move_by_k<X, ROWS_BWD>(a, s);
    return move_by_k<X, SUM_FWD>(a, s);
}

// The sum's gradients: L lanes hold a row, a vector each (rows of more than 64
// vectors in rounds), read dy once and each of its K rows of ys, write w dy in
// their places, and sum up <dy, ys>, of which a vector that moved back counts
// the channels of its own. Fewer lanes with three vectors each were slower
// (401,408 slots of 96 bf16 channels 47.5 us against 42.3; 25,088 of 384 the
// same 11.5).
template <typename X, int L, int KK, bool PART>
__device__ __forceinline__ void expert_sum_bwd_wg(const ExpertArgs& a, uint32_t G, uint64_t wg, uint32_t S,
                                                  uint32_t kept) {
    const uint64_t row = (wg * T + threadIdx.x) / L;
    const uint32_t lane = threadIdx.x % L;
    const bool in = row < (uint64_t)a.N;
    const X* dy = (const X*)a.rows + (in ? row * a.C : 0);
    const int* place = a.place + row * a.K;
    auto load = [&](Vec<X, CG>& v, const X* p, uint32_t c) {
        if constexpr (PART)
            v.load_part(p, a.C);
        else
            v.load(p + c);
    };
    for (int k = 0; k < a.K; k += KK) {
        Slot s[KK];
        float w[KK], dot[KK];
#pragma unroll
        for (int i = 0; i < KK; ++i) {
            s[i] = slot_of(in && k + i < a.K ? (uint32_t)place[k + i] : ~0u, S, kept);
            w[i] = s[i].live && a.to_sorted ? a.w[row * a.K + k + i] : 0.f;
            dot[i] = 0.f;
        }
        for (uint32_t v = lane; v < G; v += L) {
            const uint32_t c = PART ? 0 : min(v * CG, (uint32_t)a.C - CG), shared = v * CG - c;
            Vec<X, CG> d, y[KK];
            load(d, dy, c);
#pragma unroll
            for (int i = 0; i < KK; ++i)
                if (a.dw) load(y[i], (const X*)a.sorted + (s[i].live ? (size_t)s[i].at * a.C : 0), c);
#pragma unroll
            for (int i = 0; i < KK; ++i) {
                float o[CG];
#pragma unroll
                for (int j = 0; j < CG; ++j) {
                    o[j] = s[i].live ? w[i] * d[j] : 0.f;
                    const float more = fmaf(d[j], y[i][j], dot[i]);
                    dot[i] = (uint32_t)j < shared || !s[i].live ? dot[i] : more;
                }
                if (s[i].is && a.to_sorted) {
                    X* out = (X*)a.to_sorted + (size_t)s[i].at * a.C;
                    if constexpr (PART)
                        store_part<X, CG>(out, o, a.C);
                    else
                        store_vec<X, CG>(out + c, o);
                }
            }
        }
        if (a.dw) {
#pragma unroll
            for (int i = 0; i < KK; ++i) {
                const float sum = lane_sum<L>(dot[i]);
                if (lane == 0 && in && k + i < a.K) a.dw[row * a.K + k + i] = sum;
            }
        }
    }
}

template <typename X, int L, int KK, bool PART>
__global__ __launch_bounds__(T) void k_expert_sum_bwd(ExpertArgs a, uint32_t G, uint64_t wgs) {
    const uint32_t S = (uint32_t)(a.N * a.K), kept = kept_of(a);
    for (uint64_t wg = blockIdx.x; wg < wgs; wg += gridDim.x) expert_sum_bwd_wg<X, L, KK, PART>(a, G, wg, S, kept);
}

template <typename X, int L, int KK>
hipError_t sum_bwd_launch(const ExpertArgs& a, hipStream_t s) {
    const uint32_t G = (uint32_t)cdiv(a.C, CG);
    const uint64_t wgs = ((uint64_t)a.N * L + T - 1) / T;
    if constexpr (L == 4) {
        if (a.C < CG) {
            hipLaunchKernelGGL((k_expert_sum_bwd<X, L, KK, true>), dim3(grid_of(wgs)), dim3(T), 0, s, a, G, wgs);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((k_expert_sum_bwd<X, L, KK, false>), dim3(grid_of(wgs)), dim3(T), 0, s, a, G, wgs);
    return hipGetLastError();
}

// The fewest lanes that hold a row.
template <typename X, int KK>
hipError_t sum_bwd_by_row(const ExpertArgs& a, hipStream_t s) {
    const int G = cdiv(a.C, CG);
    if (G <= 4) return sum_bwd_launch<X, 4, KK>(a, s);
    if (G <= 8) return sum_bwd_launch<X, 8, KK>(a, s);
    if (G <= 16) return sum_bwd_launch<X, 16, KK>(a, s);
    if (G <= 32) return sum_bwd_launch<X, 32, KK>(a, s);
    return sum_bwd_launch<X, 64, KK>(a, s);
}

// As many slots at a time as a row has, four at most: room for more is masked
// work (200,704 rows of 96 bf16 channels with one slot 26.4 us, 30.6 with room
// for two and 35.4 for four, with two slots 41.9 and 49.2; the weighted sum 15.8,
// 16.1 and 16.5).
template <typename X>
hipError_t sum_bwd_by_k(const ExpertArgs& a, hipStream_t s) {
    if (a.K == 1) return sum_bwd_by_row<X, 1>(a, s);
    if (a.K == 2) return sum_bwd_by_row<X, 2>(a, s);
    return sum_bwd_by_row<X, 4>(a, s);
}

}  // namespace

hipError_t expert_move(const ExpertArgs& a, int op, int bf16, hipStream_t s) {
    return bf16 ? move_by_op<bf16_t>(a, op, s) : move_by_op<float>(a, op, s);
}

hipError_t expert_sum_bwd(const ExpertArgs& a, int bf16, hipStream_t s) {
    return bf16 ? sum_bwd_by_k<bf16_t>(a, s) : sum_bwd_by_k<float>(a, s);
}

}  // namespace wtc
