// The optimizer's step over many tensors: the gradients' norm and AdamW.
//
// A launch takes a table of tensors in its arguments (4 KB at most, so a long
// list is several launches). Tensors are cut into pieces of a fixed number of
// elements, one a workgroup; a workgroup finds its tensor by the numbers of
// the tensors' first workgroups.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "wtconv_device.h"

namespace wtc {

constexpr int OB = 256;            // elements of a block of the states
constexpr int ADAM_PIECE = 4096;   // elements of a workgroup

struct AdamTensor {
    void* p;
    const void* g;
    uint64_t count;
    uint32_t block;   // the tensor's first block in the states
    uint32_t wg;      // its first workgroup
    float lr, wd;
    uint32_t site;
    uint32_t pad;
};
constexpr int ADAM_TENSORS = 80;

struct AdamArgs {
    void *m, *v;
    float *scales, *master;
    const long long* step;
    const float *factor, *lr_factor;   // null: 1
    const unsigned long long* rng;
    float b1, b2, a1, a2;              // betas, 1 - betas
    float log1, log2, eps;             // log(beta)
    int n;
    AdamTensor t[ADAM_TENSORS];
};
static_assert(sizeof(AdamArgs) <= 4096, "");

enum { STATES_32 = 0, STATES_8 = 1, STATES_8_RANDOM = 2 };
hipError_t adamw_launch(const AdamArgs& a, uint32_t wgs, int p_bf16, int g_bf16, int mode, hipStream_t s);

struct NormTensor {
    const void* g;
    uint64_t count;
    uint32_t wg;
    uint32_t bf16;
};
constexpr int NORM_TENSORS = 160;

struct NormArgs {
    double* sums;       // a sum a workgroup
    uint64_t piece;     // elements of a workgroup
    int n, pad;
    NormTensor t[NORM_TENSORS];
};
static_assert(sizeof(NormArgs) <= 4096, "");

constexpr uint32_t NORM_WGS = 2048;   // most sums of a launch, besides one more a tensor
hipError_t norm_launch(const NormArgs& a, uint32_t wgs, hipStream_t s);
hipError_t norm_finish(const double* sums, uint32_t n, double max_norm, long long* step, float* out, hipStream_t s);

}  // namespace wtc
