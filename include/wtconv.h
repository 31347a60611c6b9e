/*
 * wtconv.h - C-ABI of the MI355X (gfx950) WTConv library, libwtconv.so.
 *
 * The operation
 * -------------
 * A wavelet-convolution (WTConv) layer, as named in the abstract of
 * "I/O-aware reformulation of wavelet convolution" (arXiv:2608.10805;
 * tech.sinsc.com page, Abstract, and the layerthelatestinalattice.com
 * summary): a depthwise base convolution plus an L-level Haar wavelet branch.
 * Per (b, c) plane:
 *
 *   X_0 = x;  for l = 1..L: (LL, B1, B2, B3)_l = DWT(X_{l-1}), X_l = LL_l
 *   Z_l^s = scale[l][c][s] * corr(band_l^s, w_lvl[l][c][s])        s = 0..3
 *   R_L = 0;  R_{l-1} = IWT(Z_l^0 + R_l, Z_l^1, Z_l^2, Z_l^3)
 *   y = corr(x, w_base[c]) + R_0
 *
 *   DWT on the 2x2 block (a b / c d): LL = (a+b+c+d)/2, B1 = (a+b-c-d)/2,
 *   B2 = (a-b+c-d)/2, B3 = (a-b-c+d)/2 (orthonormal); IWT is its inverse.
 *   corr(u, w)[i][j] = sum_{m,n<k} w[m][n] u[i+m-k/2][j+n-k/2], zero outside
 *   the level's own band grid (cross-correlation, 'same', stride 1).
 *   An h x w image with odd h (w) is analysed as if it had one more, zero,
 *   row (column): its bands are ceil(h/2) x ceil(w/2); IWT returns the
 *   h x w image and drops the extra row (column). Where 2^L divides H and W
 *   this is the plain halving of the pages' workloads.
 *
 * The kernels evaluate this through the three reformulations the abstract
 * lists: the Haar analysis is recomputed on chip from x (or dy) and never
 * stored, the synthesis cascade is one closed-form pass indexed by the bits of
 * the output coordinates, and the scales are folded into the convolution
 * results. The result equals the cascade up to fp32 rounding order.
 *
 * Data layout (all device pointers, caller-owned):
 *   x, y, dy, dx   [B][C][H][W] contiguous (desc->layout WTCONV_NCHW) or
 *                  [B][H][W][C] (WTCONV_NHWC), element type = desc->dtype
 *   w_base         [C][k_base][k_base]        fp32
 *   w_lvl          [L][C][4][k_level][k_level] fp32 (level index 0 = level 1)
 *   scale          [L][C][4]                  fp32
 *   gradients      fp32, same layouts as the parameters
 * Band order s: 0 LL, 1 B1 (difference across rows), 2 B2 (difference across
 * columns), 3 B3.
 *
 * Arithmetic: activations are loaded as fp32 (bf16 widened exactly), all
 * products and sums are fp32, and bf16 outputs are rounded to nearest even.
 *
 * Ownership and synchronisation: the library allocates nothing, keeps no
 * pointer after a call returns, never synchronises the stream, and is
 * reentrant. Work is enqueued on `stream` (a hipStream_t; NULL = the null
 * stream). Outputs are overwritten, never accumulated. x and y (dy and dx)
 * must not overlap.
 *
 * Errors: every argument is validated on the host before anything is
 * launched; on error nothing is enqueued and the status says why. A failed
 * launch (hipGetLastError) returns WTCONV_ERR_LAUNCH.
 */
#ifndef WTCONV_H
#define WTCONV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    WTCONV_F32 = 0,    /* fp32 activations */
    WTCONV_BF16 = 1    /* bf16 activations, fp32 arithmetic */
} wtconv_dtype_t;

typedef enum {
    WTCONV_NCHW = 0,   /* [B][C][H][W] contiguous */
    WTCONV_NHWC = 1    /* channels last: [B][H][W][C] contiguous */
} wtconv_layout_t;

typedef enum {
    WTCONV_OK = 0,
    WTCONV_ERR_INVALID_ARG = 1,        /* null pointer, overlap, bad dtype or
                                          layout, B < 0, C, H or W < 1 */
    WTCONV_ERR_UNSUPPORTED_SHAPE = 2,  /* even or unsupported k, L out of
                                          range, H*W above 2^30 (block
                                          operators: or C), B*C above
                                          2^31 - 1, or 2^32 and more dropout
                                          groups; expert rows and the
                                          optimizer: sizes past those of
                                          their descriptors */
    WTCONV_ERR_WORKSPACE = 3,          /* ws too small or misaligned */
    WTCONV_ERR_LAUNCH = 4,             /* the HIP runtime rejected a launch */
    WTCONV_ERR_SCRATCH_LIMIT = 5       /* wtconv_bwd_weight_noalloc: the call needs
                                          more than WTCONV_NOALLOC_SCRATCH_BYTES */
} wtconv_status_t;

/* Size of the static device scratch array of wtconv_bwd_weight_noalloc (one
   per GPU the library runs on, held until the process ends). */
#define WTCONV_NOALLOC_SCRATCH_BYTES (64u << 20)

typedef enum {
    WTCONV_OP_FWD = 0,
    WTCONV_OP_BWD_DATA = 1,
    WTCONV_OP_BWD_WEIGHT = 2,
    WTCONV_OP_BWD = 3          /* wtconv_bwd: both backward results */
} wtconv_op_t;

typedef struct {
    int32_t B, C, H, W;   /* activation shape, NCHW; B = 0 is an empty batch:
                             the data passes write nothing (activation
                             pointers may be NULL), the weight gradients
                             are zero */
    int32_t levels;       /* L, 0..5 */
    int32_t k_base;       /* base kernel size: odd, 1..15 */
    int32_t k_level;      /* per-level kernel size: odd, 1..15 */
    int32_t dtype;        /* wtconv_dtype_t */
    int32_t layout;       /* wtconv_layout_t of x, y, dy, dx (all four alike) */
} wtconv_desc_t;

/* Bytes of device workspace `op` needs for `desc` (0 if none). Returns
   (size_t)-1 if the descriptor is invalid or unsupported. Workspace pointers
   must be 256-byte aligned. */
size_t wtconv_workspace_size(const wtconv_desc_t *desc, int32_t op);

/* How a call of `op` (wtconv_op_t) runs for `desc`, so that a caller can
   tell a shape the fused kernels cover from one that takes the generic
   chain (same results, many times slower):
   - WTCONV_ROUTE_GENERIC: the one-kernel-per-step chain (no fused kernel
     for this shape, or an empty batch, for which nothing is launched but
     the zeroing of the weight gradients);
   - WTCONV_ROUTE_FUSED: fused kernels on the activations as they are;
   - WTCONV_ROUTE_FUSED_COPIES: fused kernels on planar copies of
     channels-last activations in the workspace;
   - WTCONV_ROUTE_SINGLE_PASS (WTCONV_OP_BWD only): one kernel reads x and
     dy once for dx and every weight gradient.
   For WTCONV_OP_BWD a shape reports FUSED (or FUSED_COPIES) when both of
   its backward passes are fused, else GENERIC. Returns -1 if the
   descriptor or op is invalid. No device call is made. */
typedef enum {
    WTCONV_ROUTE_GENERIC = 0,
    WTCONV_ROUTE_FUSED = 1,
    WTCONV_ROUTE_FUSED_COPIES = 2,
    WTCONV_ROUTE_SINGLE_PASS = 3
} wtconv_route_t;
int32_t wtconv_route(const wtconv_desc_t *desc, int32_t op);

/* Forward: y = WTConv(x). One fused pass: reads x once, writes y once.
   Workspace: wtconv_workspace_size(desc, WTCONV_OP_FWD) bytes (0 for planes
   that fit one workgroup's LDS; ws may then be NULL).
   L = 0 is the plain depthwise correlation; it has its own fused kernels
   on 56x56, 28x28 and 14x14 planes with k_base 5 or 7.
   Shapes without a fused kernel (any other H, W >= 1, L in 0..5, odd k up
   to 15) run the generic
   one-kernel-per-step chain of the naive entry points below: the same
   results and semantics, with the intermediates in the workspace, which
   wtconv_workspace_size then reports. A channels-last call of a planned
   shape converts its activations to planar copies in the workspace (after
   the kernels' own part), runs the fused kernels on them and converts the
   result back: bit for bit the planar results, two extra passes over the
   activations. The same holds for wtconv_bwd_data and wtconv_bwd_weight. */
wtconv_status_t wtconv_fwd(const wtconv_desc_t *desc, const void *x,
                           const float *w_base, const float *w_lvl,
                           const float *scale, void *y, void *ws,
                           size_t ws_bytes, void *stream);

/* Backward data: dx = J^T dy. The transpose of the layer is the same layer
   with every kernel turned by 180 degrees (the orthonormal Haar analysis and
   synthesis are each other's transpose, and corr^T is corr with the flipped
   kernel), so this runs the forward kernels with rotated weight indexing. */
wtconv_status_t wtconv_bwd_data(const wtconv_desc_t *desc, const void *dy,
                                const float *w_base, const float *w_lvl,
                                const float *scale, void *dx, void *ws,
                                size_t ws_bytes, void *stream);

/* Backward weight: with G_l^s = sum_{b,i,j} (A_l^s dy)[i][j] (A_l^s x)[i+m-p][j+n-p]
   the correlation of the two Haar pyramids (A_l^s = level-l band s analysis),
     dw_base[c]      = sum_b corr-grad(x, dy)               [C][kb][kb]
     dw_lvl[l][c][s] = scale[l][c][s] * G_l^s                [L][C][4][k][k]
     dscale[l][c][s] = sum_{m,n} w_lvl[l][c][s][m][n] * G_l^s[m][n]
   (the scale-folding reformulation applied to the gradient). The batch sum
   is a fixed-order two-stage reduction, so results are bitwise
   reproducible. Workspace: wtconv_workspace_size(desc, WTCONV_OP_BWD_WEIGHT). */
wtconv_status_t wtconv_bwd_weight(const wtconv_desc_t *desc, const void *x,
                                  const void *dy, const float *w_lvl,
                                  const float *scale, float *dw_base,
                                  float *dw_lvl, float *dscale, void *ws,
                                  size_t ws_bytes, void *stream);

/* Backward weight without allocation, for callers that cannot allocate
   device memory (code under HIP graph capture, tight serving loops, harnesses
   that forbid allocation): the same kernels, results and semantics as
   wtconv_bwd_weight (bit for bit), with the scratch that call takes as a
   workspace (per-chunk partial sums, the level-split planes, channels-last
   copies) held in a static device array of WTCONV_NOALLOC_SCRATCH_BYTES
   (64 MiB) instead. A call whose wtconv_workspace_size(desc,
   WTCONV_OP_BWD_WEIGHT) exceeds that returns WTCONV_ERR_SCRATCH_LIMIT and
   enqueues nothing (the stage-shape and 128x128 workloads fit; 16 x 256 x
   256^2 at L = 4 does not). It calls no allocating routine; its first call on
   a device looks up that device's copy of the array (hipGetSymbolAddress)
   and keeps its address. Every call on one device shares that device's
   array: calls that overlap on one GPU (on different streams, or from
   different threads, without ordering) race on it and must not be made.
   Nothing in the array needs to start at zero (every word read was written
   earlier in the same call). */
wtconv_status_t wtconv_bwd_weight_noalloc(const wtconv_desc_t *desc, const void *x,
                                          const void *dy, const float *w_lvl,
                                          const float *scale, float *dw_base,
                                          float *dw_lvl, float *dscale, void *stream);

/* Whole backward pass: dx (as wtconv_bwd_data) and the weight gradients (as
   wtconv_bwd_weight) in one call. Results equal those of the two calls bit
   for bit (the same multiply-adds in the same order), except where noted
   for the one-level single pass; what the call saves depends on the shape
   (planar layout in each case):
   - L = 0 on the planes its kernel covers (56x56, 28x28, 14x14; k_base 5 or
     7): a single pass that reads x and dy once, the fused backward the I/O
     model counts at 5*N*e instead of 6*N*e bytes per step;
   - L = 1 on 14x14 planes with 5x5 kernels: a single pass that reads x and
     dy once and computes dx and every weight gradient's partial sums in one
     kernel (then the weight gradient's fixed-order second stage); dx equals
     the two calls' bit for bit, the weight gradients group their products
     differently and agree with the two calls' to fp32 rounding (both are
     deterministic);
   - planes split into fine tiles and a coarse level-L0 image (256x256 at
     L = 4 with kernels 7 and 5, and the 64x64 test plans): the weight pass
     runs first and leaves the 2^L0-block sums of dy in the workspace; the
     backward-data pass then takes its coarse levels from those sums instead
     of reading dy a second time for them, and the weight pass's fixed-order
     second stage runs as extra workgroups of that coarse step's launch;
   - whole-plane data kernels (the stage planes, 128x128, the family of
     planes of 56, 28, 14 and 7 pixels): the weight pass runs first and the
     fixed-order second stage of its reduction runs as extra workgroups of
     the backward-data launch (one launch fewer);
   - other shapes: the two backward calls in stream order on one workspace.
   x and dy must not overlap dx. Workspace:
   wtconv_workspace_size(desc, WTCONV_OP_BWD). */
wtconv_status_t wtconv_bwd(const wtconv_desc_t *desc, const void *x,
                           const void *dy, const float *w_base,
                           const float *w_lvl, const float *scale, void *dx,
                           float *dw_base, float *dw_lvl, float *dscale,
                           void *ws, size_t ws_bytes, void *stream);

/* Naive unfused baseline (comparator only): the same three operations as a
   chain of one-kernel-per-step launches (analysis, per-level convolution,
   scale, LL add, synthesis, base convolution, final add) that keeps every
   intermediate in device memory, as the abstract describes the reference
   implementation. Same semantics and layouts as the fused entry points;
   workspace from wtconv_naive_workspace_size. Any H, W >= 1. */
size_t wtconv_naive_workspace_size(const wtconv_desc_t *desc, int32_t op);
wtconv_status_t wtconv_naive_fwd(const wtconv_desc_t *desc, const void *x,
                                 const float *w_base, const float *w_lvl,
                                 const float *scale, void *y, void *ws,
                                 size_t ws_bytes, void *stream);
wtconv_status_t wtconv_naive_bwd_data(const wtconv_desc_t *desc, const void *dy,
                                      const float *w_base, const float *w_lvl,
                                      const float *scale, void *dx, void *ws,
                                      size_t ws_bytes, void *stream);
wtconv_status_t wtconv_naive_bwd_weight(const wtconv_desc_t *desc, const void *x,
                                        const void *dy, const float *w_lvl,
                                        const float *scale, float *dw_base,
                                        float *dw_lvl, float *dscale, void *ws,
                                        size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Block operators: what a residual block needs around its WTConv mixer and
 * its matrix products. All of them work on rows: a row is the C channels of
 * one pixel (b, i, j), or of one token (H = 1, W tokens; or H = W = 1).
 *
 *   channel norm     z = (h - mean) / sqrt(var + eps)      WTCONV_NORM_LAYER
 *                    z = h / sqrt(mean(h^2) + eps)         WTCONV_NORM_RMS
 *                    y = z * weight[c] + bias[c]
 *   block residual   out = x_scale[c] * x + gate * D(v), v = z * weight + bias
 *                    of the block's output h, or v = h     WTCONV_NORM_NONE;
 *                    gate[c] (a layer scale), gate[b][c], or none
 *   counter dropout  y = D(x)
 *
 * mean and var (biased) are over the row's channels; weight, bias, gate and
 * x_scale are fp32 and each may be NULL (1, 0, 1, 1); weight and bias need a
 * norm. h and the residual stream (x, out; of the norm: y) each have their
 * own type and memory order, so a norm reads the mixer's planar output and
 * writes the channels-last rows that a linear layer takes, and the residual
 * adds such rows to a planar x, without a copy in between. All arithmetic is
 * fp32 (the variance from a second pass over the row on chip), rounded once
 * at the store.
 *
 * D keeps an element with probability 1 - T / 65536, T = floor(65536 p + 1/2), and
 * multiplies what it keeps by 65536 / (65536 - T); what it drops is zero,
 * whatever it was (p = 1 drops everything). The mask is never stored: it is
 * a function of the element's place and of rng, two 64-bit integers in
 * device memory {seed, offset}, and of the caller's site number, so the
 * backward pass makes the same mask again. A program gives each use in a
 * step its own site (below 2^31) and changes the offset between steps; as
 * rng is read on the device, a captured graph sees the new values. The bits
 * are those of Philox4x32-10 with key (seed low, seed high) and counter
 * (group, site, offset low, offset high), group = row * ceil(C/8) + c/8,
 * row = (b * H + i) * W + j, for every memory order alike: element c is kept
 * when its 16 bits (word (c%8)/2, low half for even c) are >= T. With
 * WTCONV_DROP_SAMPLE (stochastic depth) whole samples b are kept or dropped,
 * by the low half of word 0 of counter (b, site + 2^31, ...); a dropped
 * sample's h does not influence any result, nor, without a norm, does a
 * dropped element's.
 *
 * Pointers need the alignment of their element type only; outputs must not
 * overlap inputs or each other, and backward calls that may run at the same
 * time need workspaces of their own (two captured graphs, too). B = 0 writes
 * nothing but zero parameter gradients. C and H*W go up to 2^30, B*C to
 * 2^31 - 1. Gradients of parameters are summed in a fixed order (bitwise
 * reproducible) in fp32; where dout has an infinity, dgate with a bias may be
 * NaN in that channel (it is made of two sums). A channels-last side with one
 * pixel per sample (or with one channel) has the same memory order as a planar
 * one.
 * ------------------------------------------------------------------------ */
typedef enum { WTCONV_NORM_NONE = 0, WTCONV_NORM_LAYER = 1, WTCONV_NORM_RMS = 2 } wtconv_norm_t;
typedef enum {
    WTCONV_GATE_NONE = 0,      /* gate NULL */
    WTCONV_GATE_CHANNEL = 1,   /* gate [C] */
    WTCONV_GATE_SAMPLE = 2     /* gate [B][C] */
} wtconv_gate_t;
typedef enum { WTCONV_DROP_NONE = 0, WTCONV_DROP_ELEMENT = 1, WTCONV_DROP_SAMPLE = 2 } wtconv_drop_t;

typedef struct {
    int32_t B, C, H, W;
    int32_t h_dtype, h_layout;   /* the norm's x; the block's output h; dropout's x and y */
    int32_t y_dtype, y_layout;   /* the norm's y; the residual's x and out (dropout: ignored) */
    int32_t norm;                /* wtconv_norm_t */
    float eps;                   /* normal and > 0 (FLT_MIN at least) where there is a norm */
    int32_t gate;                /* wtconv_gate_t (residual only) */
    int32_t drop;                /* wtconv_drop_t (residual and dropout) */
    double p;                    /* 0..1, read where drop is not NONE */
    int32_t site;                /* 0..2^31-1, read where drop is not NONE */
} wtconv_block_desc_t;

/* Device workspace of wtconv_norm_bwd and wtconv_residual_bwd for `desc`
   (256-byte aligned; enough for every choice of wanted outputs), or
   (size_t)-1 if the descriptor is invalid. The other calls need none. */
size_t wtconv_block_workspace_size(const wtconv_block_desc_t *desc);

/* How the norm or residual of `desc` runs: WTCONV_ROUTE_FUSED (each row is
   read once and held in registers) or WTCONV_ROUTE_GENERIC (each row is read
   once per statistic: channels-last rows of more than 16,384 channels; with a
   planar side fewer than 8 or more than 2,048 channels, or fewer than four
   pixels). -1 if the descriptor is invalid. No device
   call is made. */
int32_t wtconv_block_route(const wtconv_block_desc_t *desc);

/* y = norm(x) * weight + bias. The descriptor has a norm, no gate, no drop. */
wtconv_status_t wtconv_norm_fwd(const wtconv_block_desc_t *desc, const void *x, const float *weight,
                                const float *bias, void *y, void *stream);

/* Gradients of wtconv_norm_fwd: dx [type and order of x], dweight [C],
   dbias [C]; the statistics are computed from x again. An output that is
   NULL is not computed. */
wtconv_status_t wtconv_norm_bwd(const wtconv_block_desc_t *desc, const void *x, const void *dy,
                                const float *weight, void *dx, float *dweight, float *dbias, void *ws,
                                size_t ws_bytes, void *stream);

/* out = x_scale * x + gate * D(norm(h) * weight + bias). rng (two 64-bit
   integers on the device, 8-byte aligned) may be NULL without a drop. */
wtconv_status_t wtconv_residual_fwd(const wtconv_block_desc_t *desc, const void *x, const void *h,
                                    const float *weight, const float *bias, const float *gate,
                                    const float *x_scale, const uint64_t *rng, void *out, void *stream);

/* Gradients of wtconv_residual_fwd: dx [type and order of x] (without an
   x_scale it equals dout; NULL saves the copy), dh [type and order of h],
   dweight [C], dbias [C], dgate [C] or [B][C], dx_scale [C]. An output that
   is NULL is not computed; x is read for dx_scale only (else NULL). */
wtconv_status_t wtconv_residual_bwd(const wtconv_block_desc_t *desc, const void *x, const void *h,
                                    const void *dout, const float *weight, const float *bias,
                                    const float *gate, const float *x_scale, const uint64_t *rng, void *dx,
                                    void *dh, float *dweight, float *dbias, float *dgate, float *dx_scale,
                                    void *ws, size_t ws_bytes, void *stream);

/* y = D(x), and its gradient: dx = D(dy) by the same call. */
wtconv_status_t wtconv_dropout(const wtconv_block_desc_t *desc, const void *x, const uint64_t *rng, void *y,
                               void *stream);

/* ------------------------------------------------------------------------
 * Expert rows: the rows of a block whose MLP is a set of experts, to their
 * experts and back. Row n (a pixel or token of c channels) has k slots
 * n * k + i, each with the number of an expert; a slot whose number is not
 * in 0..experts-1 goes to no expert (padding, a row over a capacity).
 *
 *   sort   order, place, offsets: the slots sorted by expert, those of one
 *          expert in their own order, those of none last. order[p] is the
 *          slot at place p, place[slot] its place, and expert e's places are
 *          offsets[e] .. offsets[e + 1] - 1 (offsets[experts]: how many
 *          slots have an expert)
 *   rows   xs[place[n][i]] = x[n]                      (none: a row of zeros)
 *   sum    y[n] = sum_i weight[n][i] * ys[place[n][i]]     (without the none)
 *
 * and their gradients: rows backward dx[n] = sum_i dxs[place[n][i]] without
 * the none; sum backward dys[place[n][i]] = weight[n][i] * dy[n] (none:
 * zeros) and dweight[n][i] = <dy[n], ys[place[n][i]]> (none: 0). What a row
 * of ys or dxs that belongs to no expert holds reaches no result.
 *
 * x, y, dx, dy are [n][c], xs, ys, dxs, dys [n * k][c], contiguous, of type
 * `dtype`; order [n * k], place [n][k], offsets [experts + 1] are int32,
 * weight and dweight [n][k] fp32. Sums over i run in order in fp32 and are
 * rounded once. A place outside 0..n*k-1 counts as none; where places are no
 * permutation, rows of xs and dys that no place names are not written.
 * Pointers need the alignment of their element type only; outputs must not
 * overlap inputs or each other. n = 0 writes zero offsets and nothing else.
 * ------------------------------------------------------------------------ */
typedef enum { WTCONV_I32 = 0, WTCONV_I64 = 1 } wtconv_index_t;

typedef struct {
    int64_t n;         /* rows; n * k up to 2^31 - 1 */
    int32_t k;         /* slots of a row, 1..1024 */
    int32_t experts;   /* 1..1024 */
    int32_t c;         /* channels, 1..2^30 (the sort does not look at it) */
    int32_t dtype;     /* wtconv_dtype_t of the rows (the sort does not look at it) */
} wtconv_expert_desc_t;

/* Device workspace of wtconv_expert_sort (256-byte aligned; 0 for few
   slots, ws may then be NULL), or (size_t)-1 if the descriptor is invalid.
   The other calls need none. Calls that may run at the same time need
   workspaces of their own (two captured graphs, too). */
size_t wtconv_expert_workspace_size(const wtconv_expert_desc_t *desc);

/* expert: [n][k] int32 or int64 (id_type, a wtconv_index_t). */
wtconv_status_t wtconv_expert_sort(const wtconv_expert_desc_t *desc, const void *expert, int32_t id_type,
                                   int32_t *order, int32_t *place, int32_t *offsets, void *ws,
                                   size_t ws_bytes, void *stream);
wtconv_status_t wtconv_expert_rows_fwd(const wtconv_expert_desc_t *desc, const void *x, const int32_t *place,
                                       const int32_t *offsets, void *xs, void *stream);
wtconv_status_t wtconv_expert_rows_bwd(const wtconv_expert_desc_t *desc, const void *dxs, const int32_t *place,
                                       const int32_t *offsets, void *dx, void *stream);
wtconv_status_t wtconv_expert_sum_fwd(const wtconv_expert_desc_t *desc, const void *ys, const float *weight,
                                      const int32_t *place, const int32_t *offsets, void *y, void *stream);
/* dys or dweight may be NULL: not computed (ys is read for dweight only,
   weight for dys only; what is not read may be NULL). */
wtconv_status_t wtconv_expert_sum_bwd(const wtconv_expert_desc_t *desc, const void *dy, const void *ys,
                                      const float *weight, const int32_t *place, const int32_t *offsets,
                                      void *dys, float *dweight, void *stream);

/* ------------------------------------------------------------------------
 * The optimizer's step over many tensors at once: the gradients' norm, and
 * AdamW with its states in 32 or in 8 bits. Tensor i has counts[i] elements
 * (contiguous, aligned to the element). The pointers of one call go into the
 * kernels' arguments: nothing is kept, and a captured graph holds them.
 *
 * Norm: out[0] = sqrt(sum of all squares), summed in 64 bits in a fixed
 * order (bitwise reproducible); out[1] = min(1, max_norm / (norm + 1e-6)),
 * and NaN where the norm is not finite. step (may be NULL) is increased by
 * one where it is.
 *
 * AdamW, with t = *step (1 for the first step; less counts as 1), f = *factor
 * (NULL: 1), r = lr[i] * *lr_factor (NULL: 1):
 *     g' = f g,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
 *     p  = p - r wd[i] p - r (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
 * Where f is not finite nothing is changed: out[1] of the norm as the factor
 * clips the gradients, and skips a step whose gradients have an infinity or
 * a NaN. (With another factor such a gradient makes its element not finite,
 * with states in 8 bits its whole block.) All arithmetic is fp32.
 *
 * The states of all tensors stand in one buffer: tensor i's begin at element
 * 256 * sum_{j < i} ceil(counts[j] / 256). What stands between a tensor's last
 * element and the next multiple of 256 is not looked at (with 8 bits it may
 * be written with zeros). state_bits = 32: m and v are fp32. state_bits = 8:
 * m and v are e4m3 bytes that hold m and sqrt(v) in units of a block of 256
 * elements, scales[block] = {max |m|, max sqrt(v)} / 448 (fp32 pairs; first
 * moments of a block whose largest is below 2^-100 are held as zero, and a
 * root that is not zero as 2^-9 units at least, so that no parameter is
 * divided by a root that was lost). The step itself uses m and v before
 * that rounding. What is rounded are the fp32 values: of a million numbers a
 * few that stand next to a border between two of 8 bits become the other one
 * than exact arithmetic gives, the same in every call. Rounding is to the
 * nearest value, or, with rng (two 64-bit integers {seed, offset} on the
 * device, as for dropout), to the value below
 * or above it with the probabilities that make the mean right: |q| becomes
 * floor(|q| / s + (u + 1/2) / 65536) s with s the distance of e4m3 numbers at
 * q and u the low (m) or high (v) 16 bits of word e % 4 of Philox4x32-10
 * with counter (e / 4, site + i, offset low, offset high) and key (seed low,
 * seed high), for element e of tensor i. The bits are those of an element
 * dropout with the same seed, offset and site: sites site .. site + n - 1 are
 * for this call alone. A moving average changes by less
 * than half a step of 8 bits in most steps: rounded to nearest it then stays
 * where it is.
 *
 * Parameters are fp32 or bf16. With master (bf16 parameters only) the step
 * works on fp32 copies of them, laid out as the states, and writes both;
 * without it a bf16 parameter is widened, changed and rounded to nearest.
 * grads[i] = NULL leaves tensor i and its states as they are. No tensor may
 * stand twice in a call or overlap another one.
 * ------------------------------------------------------------------------ */
typedef struct {
    int32_t p_dtype, g_dtype;   /* wtconv_dtype_t of all parameters, all gradients */
    int32_t state_bits;         /* 32 or 8 */
    int32_t site;               /* 0..2^31-1, read with rng: tensor i uses site + i (below 2^31) */
    double beta1, beta2;        /* 0 <= beta < 1 */
    double eps;                 /* FLT_MIN at least, finite */
} wtconv_adamw_desc_t;

#define WTCONV_ADAMW_BLOCK 256   /* elements that share a scale, and the states' alignment */

/* Elements of the states' buffers (and of master) for n tensors of these
   counts, or -1 where a count is not in 0..2^34 or the sum exceeds 2^39. */
int64_t wtconv_adamw_state_count(const int64_t *counts, int32_t n);

/* Host arrays of n entries: params, grads, counts (0..2^34 each), lr,
   weight_decay (finite); all other pointers are device memory. m, v and
   master are aligned to 16 bytes, scales to 8. */
wtconv_status_t wtconv_adamw_step(const wtconv_adamw_desc_t *desc, int32_t n, void *const *params,
                                  const void *const *grads, const int64_t *counts, const float *lr,
                                  const float *weight_decay, void *m, void *v, float *scales, float *master,
                                  const int64_t *step, const float *factor, const float *lr_factor,
                                  const uint64_t *rng, void *stream);

/* What wtconv_adamw_step returns for these arguments where it refuses them,
   and WTCONV_OK otherwise; launches nothing and makes no device call. For a
   caller whose step is several calls, all or none of which are to be made. */
wtconv_status_t wtconv_adamw_check(const wtconv_adamw_desc_t *desc, int32_t n, void *const *params,
                                   const void *const *grads, const int64_t *counts, const float *lr,
                                   const float *weight_decay, const void *m, const void *v, const float *scales,
                                   const float *master, const int64_t *step, const float *factor,
                                   const float *lr_factor, const uint64_t *rng);

/* Device workspace of wtconv_grad_norm for n tensors of these counts (8-byte
   aligned; 0 for few elements, ws may then be NULL), or (size_t)-1 where a
   count is not in 0..2^34, their sum exceeds 2^39 or n < 0. */
size_t wtconv_grad_norm_workspace_size(const int64_t *counts, int32_t n);

/* dtypes: a wtconv_dtype_t for each gradient (host array, as grads and
   counts); max_norm > 0, infinity for no clipping. out: two fp32 numbers. A
   NULL gradient counts nothing. Gradients are at addresses below 2^48, as
   the GPU's are. */
wtconv_status_t wtconv_grad_norm(int32_t n, const void *const *grads, const int64_t *counts,
                                 const int32_t *dtypes, double max_norm, int64_t *step, float *out, void *ws,
                                 size_t ws_bytes, void *stream);

/* Static description of a status code. */
const char *wtconv_status_string(wtconv_status_t status);

/* Library version, e.g. "0.5.0". */
const char *wtconv_version(void);

/* Measurement probes (not operations of the layer). They measure on the
   device the two ceilings the kernels above are compared with.
   wtconv_peak_fma: `blocks` workgroups of 256 lanes; every lane runs 16
   independent chains of `iters` unpacked fp32 FMAs and writes one float to
   out[blocks * 256] (16-byte aligned): 2 * 16 * iters * 256 * blocks flops.
   blocks and iters in 1..2^20, else WTCONV_ERR_INVALID_ARG.
   wtconv_peak_copy: copies `bytes` (a multiple of 16) from src to dst, both
   16-byte aligned and not overlapping: 2 * bytes of HBM traffic.
   Both only enqueue on `stream`; time them with events. */
wtconv_status_t wtconv_peak_fma(float *out, int32_t blocks, int32_t iters, void *stream);
wtconv_status_t wtconv_peak_copy(const void *src, void *dst, size_t bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* WTCONV_H */
