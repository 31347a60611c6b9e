// Expert rows: slots sorted by expert, rows to their experts and back.
//
// Row n has K slots n K + k, S = N K in all. place[slot] is a slot's sorted
// place; places from `offsets[E]` on belong to slots of no expert.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "wtconv_device.h"

namespace wtc {

constexpr int MAX_EXPERTS = 1024;

struct ExpertArgs {
    const void* rows;      // [N][C]: x, dy
    const void* sorted;    // [S][C]: dxs, ys
    void* to_rows;         // [N][C]: y, dx
    void* to_sorted;       // [S][C]: xs, dys (null: not wanted)
    const float* w;        // [N][K]
    float* dw;             // [N][K] (null: not wanted)
    const int* place;      // [N][K]
    const int* offsets;    // [E + 1]
    long long N;
    int K, C, E;
};

struct SortArgs {
    const void* expert;    // [S] of int32 or int64
    int* order;            // [S]
    int* place;            // [S]
    int* offsets;          // [E + 1]
    int* counts;           // of each part and expert, then totals: the workspace
    uint32_t S;
    int E, parts;
    uint32_t per;          // slots of a part
};

size_t expert_sort_bytes(long long S, int E);
hipError_t expert_sort(SortArgs a, int id64, hipStream_t s);

enum { ROWS_FWD = 0, ROWS_BWD = 1, SUM_FWD = 2 };
hipError_t expert_move(const ExpertArgs& a, int op, int bf16, hipStream_t s);
hipError_t expert_sum_bwd(const ExpertArgs& a, int bf16, hipStream_t s);

}  // namespace wtc
