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

constexpr int OB = 256;   // elements of a block of the states

// A tensor of a launch in 32 bytes: 330 tensors are three launches instead of
// five at 48. What few tensors have of their own (rate and decay) is in a
// short table beside.
struct AdamTensor {
    void* p;
    const void* g;
    uint32_t last;    // count - 1, its low 32 bits
    uint32_t block;   // the tensor's first block in the states
    uint32_t wg;      // its first workgroup
    uint32_t more;    // its number in the call, its rates', and the two high bits of count - 1
};
// Tensors of a launch; a launch of few has a short table of its own, as 4 KB of
// arguments take the host 1 us more than a hundred bytes (3.5 us against 2.5).
constexpr int ADAM_TENSORS = 119, ADAM_FEW = 16, ADAM_RATES = 16;
constexpr uint32_t ADAM_NUMBERS = 1u << 26;   // tensors of a call

struct AdamHead {
    void *m, *v;
    float *scales, *master;
    const long long* step;
    const float *factor, *lr_factor;   // null: 1
    const unsigned long long* rng;
    float b1, b2, a1, a2;              // betas, 1 - betas
    float log1, log2, eps;             // log(beta)
    uint32_t site;
    int n, rates;
    float lr[ADAM_RATES], wd[ADAM_RATES];
};
template <int N>
struct AdamTable : AdamHead {
    static constexpr int MOST = N;
    AdamTensor t[N];
};
typedef AdamTable<ADAM_TENSORS> AdamArgs;
static_assert(sizeof(AdamArgs) + 8 <= 4096, "");   // and the number of workgroups

enum { STATES_32 = 0, STATES_8 = 1, STATES_8_RANDOM = 2 };
// Blocks of a wavefront, of which a workgroup has four, and elements of a workgroup.
constexpr int adam_blocks(bool p_bf16, bool master, int mode) { return p_bf16 && !master && mode != STATES_32 ? 2 : 1; }
constexpr int adam_piece(bool p_bf16, bool master, int mode) { return 4 * OB * adam_blocks(p_bf16, master, mode); }
hipError_t adamw_launch(const AdamArgs& a, uint32_t wgs, int p_bf16, int g_bf16, int mode, hipStream_t s);

// A gradient of a launch in 12 bytes, so that one launch takes hundreds: its
// address (48 bits; even, so bit 0 says bf16), count - 1 (34 bits) and first
// workgroup (the 14 high bits of the last word).
struct NormTensor {
    uint32_t w[3];
};
constexpr int NORM_TENSORS = 339, NORM_FEW = 40;

struct NormHead {
    double* sums;       // a sum a workgroup
    uint64_t piece;     // elements of a workgroup
    int n, pad;
};
template <int N>
struct NormTable : NormHead {
    static constexpr int MOST = N;
    NormTensor t[N];
};
typedef NormTable<NORM_TENSORS> NormArgs;
static_assert(sizeof(NormArgs) <= 4096, "");

// Most sums of a launch, besides one more a tensor: fewer workgroups in all than
// the card holds at once (256 CUs, eight of four wavefronts each), as the few
// that would come after took as long as the others. 34 M bf16 elements in 330
// tensors: 18.7 us with 1,536, 21.0 with 2,048, 22.5 with 8,192.
constexpr uint32_t NORM_WGS = 1536;
static_assert(NORM_WGS + NORM_TENSORS < 1u << 14, "");
// Up to so many pieces of so many elements are one workgroup's: its table has an
// entry a piece, as above without a first workgroup.
constexpr int NORM_PIECES = 64, NORM_PIECE = 2048;
hipError_t norm_alone(const NormTable<NORM_PIECES>& a, double max_norm, long long* step, float* out, hipStream_t s);
hipError_t norm_launch(const NormArgs& a, uint32_t wgs, hipStream_t s);
hipError_t norm_finish(const double* sums, uint32_t n, double max_norm, long long* step, float* out, hipStream_t s);

}  // namespace wtc
