// C-ABI of the block operators: argument validation on the host, then
// dispatch. Nothing is launched unless every check passes.
#include <hip/hip_runtime.h>

#include <float.h>
#include <math.h>
#include <stdint.h>

#include "../../include/wtconv.h"
#include "wtconv_block.h"
#include "wtconv_buffers.h"

namespace {

using wtc::aligned;
using wtc::buffers_ok;
using wtc::done;
using wtc::elem_bytes;

size_t act_count(const wtconv_block_desc_t* d) { return (size_t)d->B * d->C * d->H * d->W; }

wtconv_status_t check_desc(const wtconv_block_desc_t* d) {
    if (!d) return WTCONV_ERR_INVALID_ARG;
    if (d->B < 0 || d->C < 1 || d->H < 1 || d->W < 1) return WTCONV_ERR_INVALID_ARG;
    for (int dt : {d->h_dtype, d->y_dtype})
        if (dt != WTCONV_F32 && dt != WTCONV_BF16) return WTCONV_ERR_INVALID_ARG;
    for (int lo : {d->h_layout, d->y_layout})
        if (lo != WTCONV_NCHW && lo != WTCONV_NHWC) return WTCONV_ERR_INVALID_ARG;
    if (d->norm < WTCONV_NORM_NONE || d->norm > WTCONV_NORM_RMS) return WTCONV_ERR_INVALID_ARG;
    // a denormal eps would leave a row of zeros an infinite reciprocal root
    if (d->norm != WTCONV_NORM_NONE && !(d->eps >= FLT_MIN && isfinite(d->eps))) return WTCONV_ERR_INVALID_ARG;
    if (d->gate < WTCONV_GATE_NONE || d->gate > WTCONV_GATE_SAMPLE) return WTCONV_ERR_INVALID_ARG;
    if (d->drop < WTCONV_DROP_NONE || d->drop > WTCONV_DROP_SAMPLE) return WTCONV_ERR_INVALID_ARG;
    if (d->drop != WTCONV_DROP_NONE && (!(d->p >= 0. && d->p <= 1.) || d->site < 0)) return WTCONV_ERR_INVALID_ARG;
    // the kernels count a plane's pixels and a row's channels in 32 bits, and
    // step past the end by up to a workgroup's share
    if (d->C > 1 << 30 || (int64_t)d->H * d->W > (1ll << 30) || (int64_t)d->B * d->C > (1ll << 31) - 1)
        return WTCONV_ERR_UNSUPPORTED_SHAPE;
    // 2^61 elements fit every product of sizes in 64 bits; a device holds far fewer
    if (d->drop == WTCONV_DROP_ELEMENT) {
        // the generator's first counter word holds the group's number
        const uint64_t groups = (uint64_t)d->H * d->W * (uint64_t)wtc::cdiv(d->C, wtc::CG);
        if (d->B > 0 && groups > (uint64_t)0xffffffffu / (uint64_t)d->B) return WTCONV_ERR_UNSUPPORTED_SHAPE;
    }
    return WTCONV_OK;
}

wtc::BlockArgs args_of(const wtconv_block_desc_t* d) {
    wtc::BlockArgs a = {};
    a.B = d->B;
    a.C = d->C;
    a.HW = d->H * d->W;
    // one pixel per sample, or one channel: both orders are the same memory
    const bool same = a.HW == 1 || a.C == 1;
    a.h_cl = same || d->h_layout == WTCONV_NHWC;
    a.y_cl = same || d->y_layout == WTCONV_NHWC;
    a.norm = d->norm;
    a.eps = d->eps;
    a.inv_c = 1.f / (float)d->C;
    a.gate_mode = d->gate;
    a.drop = wtc::DROP_NONE;
    a.keep = 1.f;
    if (d->drop != WTCONV_DROP_NONE) {
        a.thr = (uint32_t)(d->p * 65536.0 + 0.5);
        if (a.thr > 0) {   // at 0 everything is kept as it is
            a.drop = d->drop;
            a.keep = a.thr < 65536u ? 65536.f / (float)(65536u - a.thr) : 0.f;
        }
        a.site = (uint32_t)d->site;
    }
    return a;
}

// Everything that a backward call could be asked for: the workspace holds
// the sums of all of them.
size_t workspace(const wtconv_block_desc_t* d) {
    wtc::BlockArgs a = args_of(d);
    static float some;
    a.dw = a.db = a.dxs = &some;
    if (a.gate_mode != wtc::GATE_NONE) a.dg = &some;
    a.dh = &some;
    return wtc::block_bwd_workspace_bytes(a, d->h_dtype == WTCONV_BF16, d->y_dtype == WTCONV_BF16);
}

bool ws_ok(const wtconv_block_desc_t* d, const void* ws, size_t ws_bytes) {
    const size_t need = workspace(d);
    return need == 0 || (ws && aligned(ws, 256) && ws_bytes >= need);
}

}  // namespace

extern "C" {

size_t wtconv_block_workspace_size(const wtconv_block_desc_t* d) {
    return check_desc(d) == WTCONV_OK ? workspace(d) : (size_t)-1;
}

int32_t wtconv_block_route(const wtconv_block_desc_t* d) {
    if (check_desc(d) != WTCONV_OK) return -1;
    const int r = wtc::block_route(args_of(d), d->h_dtype == WTCONV_BF16, d->y_dtype == WTCONV_BF16);
    return r == wtc::BLOCK_FUSED ? WTCONV_ROUTE_FUSED : WTCONV_ROUTE_GENERIC;
}

wtconv_status_t wtconv_residual_fwd(const wtconv_block_desc_t* d, const void* x, const void* h, const float* weight,
                                    const float* bias, const float* gate, const float* x_scale, const uint64_t* rng,
                                    void* out, void* stream) {
    const wtconv_status_t st = check_desc(d);
    if (st != WTCONV_OK) return st;
    wtc::BlockArgs a = args_of(d);
    if ((weight || bias) && a.norm == wtc::NORM_NONE) return WTCONV_ERR_INVALID_ARG;
    if ((gate != nullptr) != (a.gate_mode != wtc::GATE_NONE) && d->B > 0) return WTCONV_ERR_INVALID_ARG;
    if (a.drop != wtc::DROP_NONE && !rng) return WTCONV_ERR_INVALID_ARG;
    if (d->B == 0) return WTCONV_OK;
    if (!x || !h || !out) return WTCONV_ERR_INVALID_ARG;
    const size_t eh = elem_bytes(d->h_dtype), ey = elem_bytes(d->y_dtype), n = act_count(d), c = (size_t)d->C * 4;
    const size_t gb = d->gate == WTCONV_GATE_SAMPLE ? c * d->B : c;
    if (!buffers_ok<7, 1>({{x, n * ey, ey}, {h, n * eh, eh}, {weight, c, 4}, {bias, c, 4}, {gate, gb, 4},
                           {x_scale, c, 4}, {rng, 16, 8}},
                          {{out, n * ey, ey}}))
        return WTCONV_ERR_INVALID_ARG;
    a.h = h;
    a.x = x;
    a.y = out;
    a.w = weight;
    a.b = bias;
    a.gate = gate;
    a.xs = x_scale;
    a.rng = (const unsigned long long*)rng;
    return done(wtc::block_fwd_launch(a, d->h_dtype == WTCONV_BF16, d->y_dtype == WTCONV_BF16, (hipStream_t)stream));
}

wtconv_status_t wtconv_norm_fwd(const wtconv_block_desc_t* d, const void* x, const float* weight, const float* bias,
                                void* y, void* stream) {
    const wtconv_status_t st = check_desc(d);
    if (st != WTCONV_OK) return st;
    wtc::BlockArgs a = args_of(d);
    if (a.norm == wtc::NORM_NONE || d->gate != WTCONV_GATE_NONE || d->drop != WTCONV_DROP_NONE)
        return WTCONV_ERR_INVALID_ARG;
    if (d->B == 0) return WTCONV_OK;
    if (!x || !y) return WTCONV_ERR_INVALID_ARG;
    const size_t eh = elem_bytes(d->h_dtype), ey = elem_bytes(d->y_dtype), n = act_count(d), c = (size_t)d->C * 4;
    if (!buffers_ok<3, 1>({{x, n * eh, eh}, {weight, c, 4}, {bias, c, 4}}, {{y, n * ey, ey}}))
        return WTCONV_ERR_INVALID_ARG;
    a.h = x;
    a.y = y;
    a.w = weight;
    a.b = bias;
    return done(wtc::block_fwd_launch(a, d->h_dtype == WTCONV_BF16, d->y_dtype == WTCONV_BF16, (hipStream_t)stream));
}

wtconv_status_t wtconv_residual_bwd(const wtconv_block_desc_t* d, const void* x, const void* h, const void* dout,
                                    const float* weight, const float* bias, const float* gate, const float* x_scale,
                                    const uint64_t* rng, void* dx, void* dh, float* dweight, float* dbias,
                                    float* dgate, float* dx_scale, void* ws, size_t ws_bytes, void* stream) {
    const wtconv_status_t st = check_desc(d);
    if (st != WTCONV_OK) return st;
    wtc::BlockArgs a = args_of(d);
    if ((weight || bias || dweight || dbias) && a.norm == wtc::NORM_NONE) return WTCONV_ERR_INVALID_ARG;
    if ((gate != nullptr) != (a.gate_mode != wtc::GATE_NONE) && d->B > 0) return WTCONV_ERR_INVALID_ARG;
    if (dgate && a.gate_mode == wtc::GATE_NONE) return WTCONV_ERR_INVALID_ARG;
    if (a.drop != wtc::DROP_NONE && !rng) return WTCONV_ERR_INVALID_ARG;
    if (d->B > 0 && (!h || !dout || (dx_scale && !x))) return WTCONV_ERR_INVALID_ARG;
    const size_t eh = elem_bytes(d->h_dtype), ey = elem_bytes(d->y_dtype), n = act_count(d), c = (size_t)d->C * 4;
    const size_t gb = d->gate == WTCONV_GATE_SAMPLE ? c * d->B : c;
    if (!buffers_ok<8, 7>({{x, n * ey, ey}, {h, n * eh, eh}, {dout, n * ey, ey}, {weight, c, 4}, {bias, c, 4},
                           {gate, gb, 4}, {x_scale, c, 4}, {rng, 16, 8}},
                          {{dx, n * ey, ey}, {dh, n * eh, eh}, {dweight, c, 4}, {dbias, c, 4}, {dgate, gb, 4},
                           {dx_scale, c, 4}, {ws, ws_bytes, 1}}))
        return WTCONV_ERR_INVALID_ARG;
    if (!ws_ok(d, ws, ws_bytes)) return WTCONV_ERR_WORKSPACE;
    if (d->B == 0 && d->gate == WTCONV_GATE_SAMPLE) dgate = nullptr;   // an empty [0][C]
    a.h = h;
    a.x = x;
    a.dy = dout;
    a.dx = dx;
    a.dh = dh;
    a.w = weight;
    a.b = bias;
    a.gate = gate;
    a.xs = x_scale;
    a.rng = (const unsigned long long*)rng;
    a.dw = dweight;
    a.db = dbias;
    a.dg = dgate;
    a.dxs = dx_scale;
    a.ws = (float*)ws;
    return done(wtc::block_bwd_launch(a, d->h_dtype == WTCONV_BF16, d->y_dtype == WTCONV_BF16, (hipStream_t)stream));
}

wtconv_status_t wtconv_norm_bwd(const wtconv_block_desc_t* d, const void* x, const void* dy, const float* weight,
                                void* dx, float* dweight, float* dbias, void* ws, size_t ws_bytes, void* stream) {
    if (d && (d->norm == WTCONV_NORM_NONE || d->gate != WTCONV_GATE_NONE || d->drop != WTCONV_DROP_NONE))
        return WTCONV_ERR_INVALID_ARG;
    // the residual's gradient with neither gate, drop nor x
    return wtconv_residual_bwd(d, nullptr, x, dy, weight, nullptr, nullptr, nullptr, nullptr, nullptr, dx, dweight,
                               dbias, nullptr, nullptr, ws, ws_bytes, stream);
}

wtconv_status_t wtconv_dropout(const wtconv_block_desc_t* d, const void* x, const uint64_t* rng, void* y,
                               void* stream) {
    const wtconv_status_t st = check_desc(d);
    if (st != WTCONV_OK) return st;
    if (d->drop == WTCONV_DROP_NONE || d->norm != WTCONV_NORM_NONE || d->gate != WTCONV_GATE_NONE || !rng)
        return WTCONV_ERR_INVALID_ARG;
    if (d->B == 0) return WTCONV_OK;
    if (!x || !y) return WTCONV_ERR_INVALID_ARG;
    const size_t e = elem_bytes(d->h_dtype), n = act_count(d);
    if (!buffers_ok<2, 1>({{x, n * e, e}, {rng, 16, 8}}, {{y, n * e, e}})) return WTCONV_ERR_INVALID_ARG;
    wtc::BlockArgs a = args_of(d);
    a.drop = d->drop;   // at threshold 0 the call still copies
    a.h = x;
    a.y = y;
    a.rng = (const unsigned long long*)rng;
    return done(wtc::dropout_launch(a, d->h_dtype == WTCONV_BF16, (hipStream_t)stream));
}

}  // extern "C"
