// C-ABI of the expert rows: argument validation on the host, then dispatch.
// Nothing is launched unless every check passes.
#include "wtconv_buffers.h"
#include "wtconv_experts.h"

namespace {

using wtc::buffers_ok;
using wtc::done;

wtconv_status_t check_desc(const wtconv_expert_desc_t* d, bool rows) {
    if (!d) return WTCONV_ERR_INVALID_ARG;
    if (d->n < 0 || d->k < 1 || d->experts < 1) return WTCONV_ERR_INVALID_ARG;
    if (d->k > 1024 || d->experts > wtc::MAX_EXPERTS) return WTCONV_ERR_UNSUPPORTED_SHAPE;
    // places are 32-bit numbers
    if (d->n > ((1ll << 31) - 1) / d->k) return WTCONV_ERR_UNSUPPORTED_SHAPE;
    if (!rows) return WTCONV_OK;
    if (d->c < 1 || (d->dtype != WTCONV_F32 && d->dtype != WTCONV_BF16)) return WTCONV_ERR_INVALID_ARG;
    // grids of 256 lanes, at most 64 of them and one vector of eight channels a row
    if (d->c > 1 << 30 || d->n * wtc::cdiv(d->c, 8) > (1ll << 38) || d->n > 1ll << 32) return WTCONV_ERR_UNSUPPORTED_SHAPE;
    return WTCONV_OK;
}

struct Sizes {
    size_t row, sorted, slots, offsets;   // bytes
    explicit Sizes(const wtconv_expert_desc_t* d)
        : row((size_t)d->n * d->c * wtc::elem_bytes(d->dtype)), sorted(row * d->k), slots((size_t)d->n * d->k * 4),
          offsets((size_t)(d->experts + 1) * 4) {}
};

wtc::ExpertArgs args_of(const wtconv_expert_desc_t* d, const int32_t* place, const int32_t* offsets) {
    wtc::ExpertArgs a = {};
    a.place = place;
    a.offsets = offsets;
    a.N = d->n;
    a.K = d->k;
    a.C = d->c;
    a.E = d->experts;
    return a;
}

}  // namespace

extern "C" {

size_t wtconv_expert_workspace_size(const wtconv_expert_desc_t* d) {
    if (check_desc(d, false) != WTCONV_OK) return (size_t)-1;
    return wtc::expert_sort_bytes(d->n * d->k, d->experts);
}

wtconv_status_t wtconv_expert_sort(const wtconv_expert_desc_t* d, const void* expert, int32_t id_type, int32_t* order,
                                   int32_t* place, int32_t* offsets, void* ws, size_t ws_bytes, void* stream) {
    const wtconv_status_t st = check_desc(d, false);
    if (st != WTCONV_OK) return st;
    if (id_type != WTCONV_I32 && id_type != WTCONV_I64) return WTCONV_ERR_INVALID_ARG;
    if (!offsets || (d->n > 0 && (!expert || !order || !place))) return WTCONV_ERR_INVALID_ARG;
    const size_t slots = (size_t)d->n * d->k, id = id_type == WTCONV_I64 ? 8 : 4;
    if (!buffers_ok<1, 4>({{expert, slots * id, id}},
                          {{order, slots * 4, 4}, {place, slots * 4, 4}, {offsets, (size_t)(d->experts + 1) * 4, 4},
                           {ws, ws_bytes, 1}}))
        return WTCONV_ERR_INVALID_ARG;
    const size_t need = wtc::expert_sort_bytes((long long)slots, d->experts);
    if (need && (!ws || !wtc::aligned(ws, 256) || ws_bytes < need)) return WTCONV_ERR_WORKSPACE;
    wtc::SortArgs a = {};
    a.expert = expert;
    a.order = order;
    a.place = place;
    a.offsets = offsets;
    a.counts = (int*)ws;
    a.S = (uint32_t)slots;
    a.E = d->experts;
    return done(wtc::expert_sort(a, id_type == WTCONV_I64, (hipStream_t)stream));
}

wtconv_status_t wtconv_expert_rows_fwd(const wtconv_expert_desc_t* d, const void* x, const int32_t* place,
                                       const int32_t* offsets, void* xs, void* stream) {
    const wtconv_status_t st = check_desc(d, true);
    if (st != WTCONV_OK) return st;
    if (d->n == 0) return WTCONV_OK;
    if (!x || !place || !offsets || !xs) return WTCONV_ERR_INVALID_ARG;
    const Sizes n(d);
    const size_t e = wtc::elem_bytes(d->dtype);
    if (!buffers_ok<3, 1>({{x, n.row, e}, {place, n.slots, 4}, {offsets, n.offsets, 4}}, {{xs, n.sorted, e}}))
        return WTCONV_ERR_INVALID_ARG;
    wtc::ExpertArgs a = args_of(d, place, offsets);
    a.rows = x;
    a.to_sorted = xs;
    return done(wtc::expert_move(a, wtc::ROWS_FWD, d->dtype == WTCONV_BF16, (hipStream_t)stream));
}

wtconv_status_t wtconv_expert_rows_bwd(const wtconv_expert_desc_t* d, const void* dxs, const int32_t* place,
                                       const int32_t* offsets, void* dx, void* stream) {
    const wtconv_status_t st = check_desc(d, true);
    if (st != WTCONV_OK) return st;
    if (d->n == 0) return WTCONV_OK;
    if (!dxs || !place || !offsets || !dx) return WTCONV_ERR_INVALID_ARG;
    const Sizes n(d);
    const size_t e = wtc::elem_bytes(d->dtype);
    if (!buffers_ok<3, 1>({{dxs, n.sorted, e}, {place, n.slots, 4}, {offsets, n.offsets, 4}}, {{dx, n.row, e}}))
        return WTCONV_ERR_INVALID_ARG;
    wtc::ExpertArgs a = args_of(d, place, offsets);
    a.sorted = dxs;
    a.to_rows = dx;
    return done(wtc::expert_move(a, wtc::ROWS_BWD, d->dtype == WTCONV_BF16, (hipStream_t)stream));
}

wtconv_status_t wtconv_expert_sum_fwd(const wtconv_expert_desc_t* d, const void* ys, const float* weight,
                                      const int32_t* place, const int32_t* offsets, void* y, void* stream) {
    const wtconv_status_t st = check_desc(d, true);
    if (st != WTCONV_OK) return st;
    if (d->n == 0) return WTCONV_OK;
    if (!ys || !weight || !place || !offsets || !y) return WTCONV_ERR_INVALID_ARG;
    const Sizes n(d);
    const size_t e = wtc::elem_bytes(d->dtype);
    if (!buffers_ok<4, 1>({{ys, n.sorted, e}, {weight, n.slots, 4}, {place, n.slots, 4}, {offsets, n.offsets, 4}},
                          {{y, n.row, e}}))
        return WTCONV_ERR_INVALID_ARG;
    wtc::ExpertArgs a = args_of(d, place, offsets);
    a.sorted = ys;
    a.w = weight;
    a.to_rows = y;
    return done(wtc::expert_move(a, wtc::SUM_FWD, d->dtype == WTCONV_BF16, (hipStream_t)stream));
}

wtconv_status_t wtconv_expert_sum_bwd(const wtconv_expert_desc_t* d, const void* dy, const void* ys,
                                      const float* weight, const int32_t* place, const int32_t* offsets, void* dys,
                                      float* dweight, void* stream) {
    const wtconv_status_t st = check_desc(d, true);
    if (st != WTCONV_OK) return st;
    if (d->n == 0 || (!dys && !dweight)) return WTCONV_OK;
    if (!dy || !place || !offsets || (dweight && !ys) || (dys && !weight)) return WTCONV_ERR_INVALID_ARG;
    const Sizes n(d);
    const size_t e = wtc::elem_bytes(d->dtype);
    if (!buffers_ok<5, 2>({{dy, n.row, e}, {dweight ? ys : nullptr, n.sorted, e}, {dys ? weight : nullptr, n.slots, 4},
                           {place, n.slots, 4}, {offsets, n.offsets, 4}},
                          {{dys, n.sorted, e}, {dweight, n.slots, 4}}))
        return WTCONV_ERR_INVALID_ARG;
    wtc::ExpertArgs a = args_of(d, place, offsets);
    a.rows = dy;
    a.sorted = ys;
    a.w = weight;
    a.to_sorted = dys;
    a.dw = dweight;
    return done(wtc::expert_sum_bwd(a, d->dtype == WTCONV_BF16, (hipStream_t)stream));
}

}  // extern "C"
