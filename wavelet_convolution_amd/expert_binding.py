"""Binding of the expert rows (argument marshalling only).

Slots sorted by expert, rows to their experts and back, as defined in
wtconv.h. Rows are tensors [..., C], contiguous; a routing's `place` is
[..., K] with the same leading dimensions (N rows in all) and its `offsets`
[E + 1], as wtconv_expert_sort returns them. Every function checks what the
plain pointers of the C ABI cannot carry and calls the C-ABI entry point of
the same name on the current stream of the tensors' device (or on `stream`,
on which outputs are then allocated too). There is no fallback.
"""
from __future__ import annotations

from . import binding as _b
from .block_binding import _elsewhere, _enter, _wanted


def wtconv_expert_sort(expert, experts: int, *, order=None, place=None, offsets=None, ws=None, stream=None):
    """(order, place, offsets), int32, of slots with experts `expert` [..., K] (int32 or int64; a number outside
    0..experts-1 is no expert): order [N * K] lists the slots (row * K + k) sorted by expert, each expert's in their
    own order and those of none last, place (expert's shape) is each slot's place in it, and expert e's places are
    offsets[e] .. offsets[e + 1] - 1 (offsets[1:] are the ends that a grouped product takes)."""
    if stream is None or not _elsewhere(expert, stream):
        r = _b.load_native().expert_sort(expert, experts, order, place, offsets, ws)
        if r is not NotImplemented:
            return r
    return _enter(wtconv_expert_sort, expert, stream, (expert, order, place, offsets, ws), expert, experts,
                  order=order, place=place, offsets=offsets, ws=ws)


def wtconv_expert_rows_fwd(x, place, offsets, *, xs=None, stream=None):
    """xs [N * K, C]: row place[n, k] is row n of x [..., C]; rows of slots without an expert are zeros."""
    if stream is None or not _elsewhere(x, stream):
        r = _b.load_native().expert_rows_fwd(x, place, offsets, xs)
        if r is not NotImplemented:
            return r
    return _enter(wtconv_expert_rows_fwd, x, stream, (x, place, offsets, xs), x, place, offsets, xs=xs)


def wtconv_expert_rows_bwd(dxs, place, offsets, *, dx=None, stream=None):
    """dx [..., C] of wtconv_expert_rows_fwd: the sum of each row's slots' rows of dxs [N * K, C]."""
    if stream is None or not _elsewhere(dxs, stream):
        r = _b.load_native().expert_rows_bwd(dxs, place, offsets, dx)
        if r is not NotImplemented:
            return r
    return _enter(wtconv_expert_rows_bwd, dxs, stream, (dxs, place, offsets, dx), dxs, place, offsets, dx=dx)


def wtconv_expert_sum_fwd(ys, weight, place, offsets, *, y=None, stream=None):
    """y [..., C]: the sum over each row's slots of weight (place's shape, fp32) times the slot's row of ys
    [N * K, C]. Slots without an expert count nothing, whatever their weight and their row of ys hold."""
    if stream is None or not _elsewhere(ys, stream):
        r = _b.load_native().expert_sum_fwd(ys, weight, place, offsets, y)
        if r is not NotImplemented:
            return r
    return _enter(wtconv_expert_sum_fwd, ys, stream, (ys, weight, place, offsets, y), ys, weight, place, offsets, y=y)


def wtconv_expert_sum_bwd(dy, ys, weight, place, offsets, *, want=("dys", "dweight"), dys=None, dweight=None,
                          stream=None):
    """(dys, dweight) of wtconv_expert_sum_fwd: rows weight * dy for the slots, zeros for those without an expert,
    and the products <dy, ys>. `want`: the names of the gradients to compute; the others are None. ys is read for
    dweight only and weight for dys only: what is not read may be None."""
    wants = _wanted(want, ("dys", "dweight"))
    if stream is None or not _elsewhere(dy, stream):
        r = _b.load_native().expert_sum_bwd(dy, ys, weight, place, offsets, *wants, dys, dweight)
        if r is not NotImplemented:
            return r
    return _enter(wtconv_expert_sum_bwd, dy, stream, (dy, ys, weight, place, offsets, dys, dweight), dy, ys, weight,
                  place, offsets, want=want, dys=dys, dweight=dweight)
