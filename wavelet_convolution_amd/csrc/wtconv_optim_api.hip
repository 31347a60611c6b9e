// C-ABI of the optimizer's step: argument validation on the host, tables of
// tensors, launches. Nothing is launched unless every check passes.
#include <float.h>
#include <math.h>
#include <stdlib.h>

#include <algorithm>

#include "wtconv_buffers.h"
#include "wtconv_optim.h"

namespace {

using wtc::aligned;
using wtc::done;
using wtc::elem_bytes;

constexpr int64_t MOST = 1ll << 34;   // elements of a tensor: the generator's first word counts them in fours
constexpr int64_t MOST_ALL = 1ll << 39;

int64_t blocks_of(int64_t count) { return (count + wtc::OB - 1) / wtc::OB; }

int64_t state_count(const int64_t* counts, int32_t n) {
    if (n < 0 || (n > 0 && !counts)) return -1;
    int64_t all = 0;
    for (int i = 0; i < n; ++i) {
        if (counts[i] < 0 || counts[i] > MOST) return -1;
        all += blocks_of(counts[i]) * wtc::OB;
        if (all > MOST_ALL) return -1;
    }
    return all;
}

// Memory of a call, sorted by its begin: an output must not overlap anything.
struct Range {
    uintptr_t begin, end;
    bool out;
};
bool disjoint(Range* r, size_t n) {
    std::sort(r, r + n, [](const Range& a, const Range& b) { return a.begin < b.begin; });
    uintptr_t any = 0, out = 0;   // ends so far
    for (size_t i = 0; i < n; ++i) {
        if (r[i].begin < out || (r[i].out && r[i].begin < any)) return false;
        any = std::max(any, r[i].end);
        if (r[i].out) out = std::max(out, r[i].end);
    }
    return true;
}
struct Ranges {
    Range few[160], *r;
    size_t n = 0;
    explicit Ranges(size_t most) : r(most <= 160 ? few : (Range*)malloc(most * sizeof(Range))) {}
    ~Ranges() {
        if (r != few) free(r);
    }
    void add(const void* p, uint64_t bytes, bool out) {
        if (p && bytes) r[n++] = {(uintptr_t)p, (uintptr_t)p + bytes, out};
    }
};

bool dtype_ok(int d) { return d == WTCONV_F32 || d == WTCONV_BF16; }

// Everything that a step refuses; whether it has something to do.
wtconv_status_t check_adamw(const wtconv_adamw_desc_t* d, int32_t n, void* const* params,
                            const void* const* grads, const int64_t* counts, const float* lr,
                            const float* weight_decay, const void* m, const void* v, const float* scales,
                            const float* master, const int64_t* step, const float* factor, const float* lr_factor,
                            const uint64_t* rng, bool& work) {
    work = false;
    if (!d || n < 0) return WTCONV_ERR_INVALID_ARG;
    if (!dtype_ok(d->p_dtype) || !dtype_ok(d->g_dtype)) return WTCONV_ERR_INVALID_ARG;
    if (d->state_bits != 8 && d->state_bits != 32) return WTCONV_ERR_INVALID_ARG;
    for (double b : {d->beta1, d->beta2})
        if (!(b >= 0. && b < 1.)) return WTCONV_ERR_INVALID_ARG;
    if (!((float)d->eps >= FLT_MIN && isfinite((float)d->eps))) return WTCONV_ERR_INVALID_ARG;
    const bool eight = d->state_bits == 8, bf16 = d->p_dtype == WTCONV_BF16;
    if (rng && (!eight || d->site < 0 || n > (1ll << 31) - d->site)) return WTCONV_ERR_INVALID_ARG;
    if (n > (int32_t)wtc::ADAM_NUMBERS) return WTCONV_ERR_UNSUPPORTED_SHAPE;
    if (n == 0) return WTCONV_OK;
    if (!params || !grads || !counts || !lr || !weight_decay || !step) return WTCONV_ERR_INVALID_ARG;
    const int64_t all = state_count(counts, n);
    if (all < 0) return WTCONV_ERR_UNSUPPORTED_SHAPE;
    if (all > 0 && (!m || !v || eight != (scales != nullptr))) return WTCONV_ERR_INVALID_ARG;
    if (master && !bf16) return WTCONV_ERR_INVALID_ARG;
    if (!aligned(m, 16) || !aligned(v, 16) || !aligned(master, 16) || !aligned(scales, 8) || !aligned(step, 8) ||
        !aligned(factor, 4) || !aligned(lr_factor, 4) || !aligned(rng, 8))
        return WTCONV_ERR_INVALID_ARG;
    const size_t ep = elem_bytes(d->p_dtype), eg = elem_bytes(d->g_dtype), es = eight ? 1 : 4;
    Ranges ranges(2 * (size_t)n + 8);
    if (!ranges.r) return WTCONV_ERR_LAUNCH;   // no host memory
    for (int i = 0; i < n; ++i) {
        if (!isfinite(lr[i]) || !isfinite(weight_decay[i])) return WTCONV_ERR_INVALID_ARG;
        if (!grads[i] || counts[i] == 0) continue;
        if (!params[i] || !aligned(params[i], ep) || !aligned(grads[i], eg)) return WTCONV_ERR_INVALID_ARG;
        ranges.add(params[i], (uint64_t)counts[i] * ep, true);
        ranges.add(grads[i], (uint64_t)counts[i] * eg, false);
    }
    if (ranges.n == 0) return WTCONV_OK;
    ranges.add(m, all * es, true);
    ranges.add(v, all * es, true);
    ranges.add(scales, all / wtc::OB * 8, true);
    ranges.add(master, all * 4, true);
    ranges.add(step, 8, false);
    ranges.add(factor, 4, false);
    ranges.add(lr_factor, 4, false);
    ranges.add(rng, 16, false);
    if (!disjoint(ranges.r, ranges.n)) return WTCONV_ERR_INVALID_ARG;
    work = true;
    return WTCONV_OK;
}

}  // namespace

extern "C" {

int64_t wtconv_adamw_state_count(const int64_t* counts, int32_t n) { return state_count(counts, n); }

wtconv_status_t wtconv_adamw_check(const wtconv_adamw_desc_t* d, int32_t n, void* const* params,
                                   const void* const* grads, const int64_t* counts, const float* lr,
                                   const float* weight_decay, const void* m, const void* v, const float* scales,
                                   const float* master, const int64_t* step, const float* factor,
                                   const float* lr_factor, const uint64_t* rng) {
    bool work;
    return check_adamw(d, n, params, grads, counts, lr, weight_decay, m, v, scales, master, step, factor, lr_factor,
                       rng, work);
}

wtconv_status_t wtconv_adamw_step(const wtconv_adamw_desc_t* d, int32_t n, void* const* params,
                                  const void* const* grads, const int64_t* counts, const float* lr,
                                  const float* weight_decay, void* m, void* v, float* scales, float* master,
                                  const int64_t* step, const float* factor, const float* lr_factor,
                                  const uint64_t* rng, void* stream) {
    bool work;
    const wtconv_status_t st = check_adamw(d, n, params, grads, counts, lr, weight_decay, m, v, scales, master, step,
                                           factor, lr_factor, rng, work);
    if (st != WTCONV_OK || !work) return st;
    const bool eight = d->state_bits == 8, bf16 = d->p_dtype == WTCONV_BF16;

    wtc::AdamArgs a = {};
    a.m = m;
    a.v = v;
    a.scales = scales;
    a.master = master;
    a.step = (const long long*)step;
    a.factor = factor;
    a.lr_factor = lr_factor;
    a.rng = (const unsigned long long*)rng;
    a.b1 = (float)d->beta1;
    a.b2 = (float)d->beta2;
    a.a1 = (float)(1. - d->beta1);
    a.a2 = (float)(1. - d->beta2);
    a.log1 = (float)log(d->beta1);   // minus infinity for 0
    a.log2 = (float)log(d->beta2);
    a.eps = (float)d->eps;
    a.site = (uint32_t)d->site;
    const int mode = !eight ? wtc::STATES_32 : rng ? wtc::STATES_8_RANDOM : wtc::STATES_8;
    const int piece = wtc::adam_piece(bf16, master != nullptr, mode);
    uint32_t wgs = 0;
    int64_t block = 0;
    auto flush = [&]() {
        const hipError_t err = a.n ? wtc::adamw_launch(a, wgs, bf16, d->g_dtype == WTCONV_BF16, mode,
                                                       (hipStream_t)stream)
                                   : hipSuccess;
        a.n = a.rates = 0;
        wgs = 0;
        return err;
    };
    // the place of a tensor's rates in the launch's table; its length where there is no room
    auto rates_of = [&](int i) {
        for (int r = a.rates - 1; r >= 0; --r)
            if (a.lr[r] == lr[i] && a.wd[r] == weight_decay[i]) return r;
        if (a.rates < wtc::ADAM_RATES) {
            a.lr[a.rates] = lr[i];
            a.wd[a.rates] = weight_decay[i];
            return a.rates++;
        }
        return wtc::ADAM_RATES;
    };
    for (int i = 0; i < n; ++i) {
        if (grads[i] && counts[i] > 0) {
            const uint32_t more = (uint32_t)((counts[i] + piece - 1) / piece);   // 2^24 at most
            int r = rates_of(i);
            if (a.n == wtc::ADAM_TENSORS || wgs + more > 1u << 30 || r == wtc::ADAM_RATES) {
                if (const hipError_t err = flush(); err != hipSuccess) return done(err);
                r = rates_of(i);
            }
            const uint64_t last = (uint64_t)counts[i] - 1;
            a.t[a.n++] = {params[i], grads[i], (uint32_t)last, (uint32_t)block, wgs,
                          (uint32_t)i | (uint32_t)r << 26 | (uint32_t)(last >> 32) << 30};
            wgs += more;
        }
        block += blocks_of(counts[i]);
    }
    return done(flush());
}

size_t wtconv_grad_norm_workspace_size(const int64_t* counts, int32_t n) {
    if (state_count(counts, n) < 0) return (size_t)-1;
    // few elements: pieces of them in one launch, whichever gradients are missing
    int64_t pieces = 0;
    for (int i = 0; i < n && pieces <= wtc::NORM_PIECES; ++i) pieces += (counts[i] + wtc::NORM_PIECE - 1) / wtc::NORM_PIECE;
    if (pieces <= wtc::NORM_PIECES) return 0;
    const size_t launches = ((size_t)n + wtc::NORM_TENSORS - 1) / wtc::NORM_TENSORS;
    return (launches * wtc::NORM_WGS + n) * sizeof(double);
}

wtconv_status_t wtconv_grad_norm(int32_t n, const void* const* grads, const int64_t* counts, const int32_t* dtypes,
                                 double max_norm, int64_t* step, float* out, void* ws, size_t ws_bytes, void* stream) {
    if (n < 0 || !out || !(max_norm > 0.)) return WTCONV_ERR_INVALID_ARG;
    if (n > 0 && (!grads || !counts || !dtypes)) return WTCONV_ERR_INVALID_ARG;
    if (!aligned(out, 4) || !aligned(step, 8)) return WTCONV_ERR_INVALID_ARG;
    const size_t need = wtconv_grad_norm_workspace_size(counts, n);
    if (need == (size_t)-1) return WTCONV_ERR_UNSUPPORTED_SHAPE;
    if (need && (!ws || !aligned(ws, 8) || ws_bytes < need)) return WTCONV_ERR_WORKSPACE;
    auto hit = [](const void* p, uint64_t np, const void* q, uint64_t nq) {
        return p && q && (uintptr_t)p < (uintptr_t)q + nq && (uintptr_t)q < (uintptr_t)p + np;
    };
    if (hit(out, 8, step, 8) || hit(out, 8, ws, need) || hit(step, 8, ws, need)) return WTCONV_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        if (!dtype_ok(dtypes[i])) return WTCONV_ERR_INVALID_ARG;
        if (!grads[i] || counts[i] == 0) continue;
        const size_t e = elem_bytes(dtypes[i]);
        const uint64_t bytes = (uint64_t)counts[i] * e;
        if (!aligned(grads[i], e) || (uint64_t)(uintptr_t)grads[i] >> 48 || hit(grads[i], bytes, out, 8) || hit(grads[i], bytes, step, 8) ||
            hit(grads[i], bytes, ws, need))
            return WTCONV_ERR_INVALID_ARG;
    }
    if (need == 0) {
        wtc::NormTable<wtc::NORM_PIECES> few = {};
        for (int i = 0; i < n; ++i)
            for (int64_t at = 0; grads[i] && at < counts[i]; at += wtc::NORM_PIECE) {
                const uint64_t g = ((uintptr_t)grads[i] + at * elem_bytes(dtypes[i])) | (dtypes[i] == WTCONV_BF16);
                const uint32_t last = (uint32_t)std::min<int64_t>(wtc::NORM_PIECE, counts[i] - at) - 1;
                few.t[few.n++] = {{(uint32_t)g, (uint32_t)(g >> 32) | last << 16, 0}};
            }
        return done(wtc::norm_alone(few, max_norm, (long long*)step, out, (hipStream_t)stream));
    }
    double* sums = (double*)ws;
    for (int at = 0; at < n;) {
        wtc::NormArgs a = {};
        int first = at;
        uint64_t all = 0;
        for (; at < n && a.n < wtc::NORM_TENSORS; ++at)
            if (grads[at] && counts[at] > 0) {
                ++a.n;
                all += (uint64_t)counts[at];
            }
        // whole rounds of vectors; at most NORM_WGS pieces, and a started one a tensor
        a.piece = std::max<uint64_t>(8192, (all / wtc::NORM_WGS + 2048) / 2048 * 2048);
        a.sums = sums;
        uint32_t wgs = 0;
        a.n = 0;
        for (; first < at; ++first)
            if (grads[first] && counts[first] > 0) {
                const uint64_t g = (uintptr_t)grads[first] | (dtypes[first] == WTCONV_BF16),
                               last = (uint64_t)counts[first] - 1;
                a.t[a.n++] = {{(uint32_t)g, (uint32_t)(g >> 32) | (uint32_t)last << 16,
                               (uint32_t)(last >> 16) | wgs << 18}};
                wgs += (uint32_t)(((uint64_t)counts[first] + a.piece - 1) / a.piece);
            }
        if (a.n == 0) continue;
        if (const hipError_t err = wtc::norm_launch(a, wgs, (hipStream_t)stream); err != hipSuccess) return done(err);
        sums += wgs;
    }
    return done(wtc::norm_finish((const double*)ws, (uint32_t)(sums - (double*)ws), max_norm, (long long*)step, out,
                                 (hipStream_t)stream));
}

}  // extern "C"
