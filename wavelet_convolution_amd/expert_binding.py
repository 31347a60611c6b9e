"""Thin ctypes binding of the expert rows (argument marshalling only).

Slots sorted by expert, rows to their experts and back, as defined in
wtconv.h. Rows are tensors [..., C], contiguous; a routing's `place` is
[..., K] with the same leading dimensions (N rows in all) and its `offsets`
[E + 1], as wtconv_expert_sort returns them. Every function checks what the
plain pointers of the C ABI cannot carry and calls the C-ABI entry point of
the same name on the current stream of the tensors' device (or on `stream`,
on which outputs are then allocated too). There is no fallback.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as _b
from .block_binding import _DTYPES, _elsewhere, _enter, _on_gpu, _stream, _wanted

_IDS = {torch.int32: 0, torch.int64: 1}


def _dense(name: str, t: torch.Tensor, dtype, shape) -> None:
    if t.dtype is not dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}; got {tuple(t.shape)} "
                         f"{t.dtype}{'' if t.is_contiguous() else ', not contiguous'}")


def _rows(name: str, t: torch.Tensor) -> int:
    """The dtype code of a tensor of rows."""
    dt = _DTYPES.get(t.dtype)
    if dt is None or t.dim() < 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 or bfloat16 tensor of rows [..., C]; got "
                         f"{tuple(t.shape)} {t.dtype}{'' if t.is_contiguous() else ', not contiguous'}")
    return dt


def _route(place: torch.Tensor, offsets: torch.Tensor, rows: torch.Tensor, dtype: int, c: int):
    """The descriptor of a call with this routing."""
    if place.dtype is not torch.int32 or place.dim() < 2 or not place.is_contiguous():
        raise ValueError(f"place must be a contiguous int32 tensor [..., K]; got {tuple(place.shape)} {place.dtype}")
    if offsets.dtype is not torch.int32 or offsets.dim() != 1 or offsets.numel() < 2 or not offsets.is_contiguous():
        raise ValueError(f"offsets must be a contiguous int32 tensor [E + 1]; got {tuple(offsets.shape)} "
                         f"{offsets.dtype}")
    k, experts = place.shape[-1], offsets.numel() - 1
    if k < 1 or c < 1:
        raise ValueError(f"a routing has at least one slot a row, and a row one channel; got K = {k}, C = {c}")
    if (k | experts | c) >> 31:
        _b._check_i32(k, experts, c)
    return _b.WTConvExpertDesc(place.numel() // k, k, experts, c, dtype)


def _sorted_rows(name: str, t: torch.Tensor, place: torch.Tensor) -> int:
    dt = _rows(name, t)
    if t.dim() != 2 or t.shape[0] != place.numel():
        raise ValueError(f"{name} must have one row a slot, ({place.numel()}, C); got {tuple(t.shape)}")
    return dt


def _token_rows(name: str, t: torch.Tensor, place: torch.Tensor) -> int:
    dt = _rows(name, t)
    if t.shape[:-1] != place.shape[:-1]:
        raise ValueError(f"{name} must have place's rows, {tuple(place.shape[:-1])} + (C,); got {tuple(t.shape)}")
    return dt


def _out(name: str, out, like: torch.Tensor, shape) -> torch.Tensor:
    """The output to write: the one given, checked, or a new one."""
    if out is None:
        return like.new_empty(shape)
    _dense(name, out, like.dtype, shape)
    return out


def wtconv_expert_sort(expert, experts: int, *, order=None, place=None, offsets=None, ws=None, stream=None):
    """(order, place, offsets), int32, of slots with experts `expert` [..., K] (int32 or int64; a number outside
    0..experts-1 is no expert): order [N * K] lists the slots (row * K + k) sorted by expert, each expert's in their
    own order and those of none last, place (expert's shape) is each slot's place in it, and expert e's places are
    offsets[e] .. offsets[e + 1] - 1 (offsets[1:] are the ends that a grouped product takes)."""
    _on_gpu(expert, order=order, place=place, offsets=offsets, ws=ws)
    if _elsewhere(expert, stream):
        return _enter(wtconv_expert_sort, expert, stream, (expert, order, place, offsets, ws), expert, experts,
                      order=order, place=place, offsets=offsets, ws=ws)
    ids = _IDS.get(expert.dtype)
    if ids is None or expert.dim() < 2 or not expert.is_contiguous():
        raise ValueError(f"expert must be a contiguous int32 or int64 tensor [..., K]; got {tuple(expert.shape)} "
                         f"{expert.dtype}{'' if expert.is_contiguous() else ', not contiguous'}")
    k, slots, experts = expert.shape[-1], expert.numel(), int(experts)
    if k < 1:
        raise ValueError("a row has at least one slot")
    if (k | experts) >> 31:
        _b._check_i32(k, experts)
    d = _b.WTConvExpertDesc(slots // k, k, experts, 0, 0)
    lib = _b.load_library()
    need = lib.wtconv_expert_workspace_size(ctypes.byref(d))
    if need == _NO_SIZE:   # the call itself says what is wrong, before it looks at a pointer
        _b._check(lib.wtconv_expert_sort(ctypes.byref(d), 0, ids, 0, 0, 0, 0, 0, 0))
    i32 = dict(dtype=torch.int32, device=expert.device)
    if order is None:
        order = torch.empty(slots, **i32)
    else:
        _dense("order", order, torch.int32, (slots,))
    if place is None:
        place = torch.empty(expert.shape, **i32)
    else:
        _dense("place", place, torch.int32, expert.shape)
    if offsets is None:
        offsets = torch.empty(experts + 1, **i32)
    else:
        _dense("offsets", offsets, torch.int32, (experts + 1,))
    if ws is None and need:
        ws = torch.empty(need + 256, dtype=torch.uint8, device=expert.device)
    _b._check(lib.wtconv_expert_sort(ctypes.byref(d), expert.data_ptr(), ids, order.data_ptr(), place.data_ptr(),
                                     offsets.data_ptr(), _b._ws_ptr(ws), _b._ws_bytes(ws), _stream(expert)))
    return order, place, offsets


_NO_SIZE = ctypes.c_size_t(-1).value


def wtconv_expert_rows_fwd(x, place, offsets, *, xs=None, stream=None):
    """xs [N * K, C]: row place[n, k] is row n of x [..., C]; rows of slots without an expert are zeros."""
    _on_gpu(x, place=place, offsets=offsets, xs=xs)
    if _elsewhere(x, stream):
        return _enter(wtconv_expert_rows_fwd, x, stream, (x, place, offsets, xs), x, place, offsets, xs=xs)
    d = _route(place, offsets, x, _token_rows("x", x, place), x.shape[-1])
    xs = _out("xs", xs, x, (place.numel(), x.shape[-1]))
    _b._check(_b.load_library().wtconv_expert_rows_fwd(ctypes.byref(d), x.data_ptr(), place.data_ptr(),
                                                       offsets.data_ptr(), xs.data_ptr(), _stream(x)))
    return xs


def wtconv_expert_rows_bwd(dxs, place, offsets, *, dx=None, stream=None):
    """dx [..., C] of wtconv_expert_rows_fwd: the sum of each row's slots' rows of dxs [N * K, C]."""
    _on_gpu(dxs, place=place, offsets=offsets, dx=dx)
    if _elsewhere(dxs, stream):
        return _enter(wtconv_expert_rows_bwd, dxs, stream, (dxs, place, offsets, dx), dxs, place, offsets, dx=dx)
    d = _route(place, offsets, dxs, _sorted_rows("dxs", dxs, place), dxs.shape[-1])
    dx = _out("dx", dx, dxs, (*place.shape[:-1], dxs.shape[-1]))
    _b._check(_b.load_library().wtconv_expert_rows_bwd(ctypes.byref(d), dxs.data_ptr(), place.data_ptr(),
                                                       offsets.data_ptr(), dx.data_ptr(), _stream(dxs)))
    return dx


def wtconv_expert_sum_fwd(ys, weight, place, offsets, *, y=None, stream=None):
    """y [..., C]: the sum over each row's slots of weight (place's shape, fp32) times the slot's row of ys
    [N * K, C]. Slots without an expert count nothing, whatever their weight and their row of ys hold."""
    _on_gpu(ys, weight=weight, place=place, offsets=offsets, y=y)
    if _elsewhere(ys, stream):
        return _enter(wtconv_expert_sum_fwd, ys, stream, (ys, weight, place, offsets, y), ys, weight, place, offsets,
                      y=y)
    d = _route(place, offsets, ys, _sorted_rows("ys", ys, place), ys.shape[-1])
    _dense("weight", weight, torch.float32, place.shape)
    y = _out("y", y, ys, (*place.shape[:-1], ys.shape[-1]))
    _b._check(_b.load_library().wtconv_expert_sum_fwd(ctypes.byref(d), ys.data_ptr(), weight.data_ptr(),
                                                      place.data_ptr(), offsets.data_ptr(), y.data_ptr(), _stream(ys)))
    return y


def wtconv_expert_sum_bwd(dy, ys, weight, place, offsets, *, want=("dys", "dweight"), dys=None, dweight=None,
                          stream=None):
    """(dys, dweight) of wtconv_expert_sum_fwd: rows weight * dy for the slots, zeros for those without an expert,
    and the products <dy, ys>. `want`: the names of the gradients to compute; the others are None."""
    _on_gpu(dy, ys=ys, weight=weight, place=place, offsets=offsets, dys=dys, dweight=dweight)
    if _elsewhere(dy, stream):
        return _enter(wtconv_expert_sum_bwd, dy, stream, (dy, ys, weight, place, offsets, dys, dweight), dy, ys,
                      weight, place, offsets, want=want, dys=dys, dweight=dweight)
    d = _route(place, offsets, dy, _token_rows("dy", dy, place), dy.shape[-1])
    slots, c = place.numel(), dy.shape[-1]
    _dense("ys", ys, dy.dtype, (slots, c))
    _dense("weight", weight, torch.float32, place.shape)
    wants = _wanted(want, ("dys", "dweight"))
    dys = _out("dys", dys, dy, (slots, c)) if wants[0] else None
    dweight = _out("dweight", dweight, weight, place.shape) if wants[1] else None
    _b._check(_b.load_library().wtconv_expert_sum_bwd(
        ctypes.byref(d), dy.data_ptr(), ys.data_ptr(), weight.data_ptr(), place.data_ptr(), offsets.data_ptr(),
        _b._ptr(dys), _b._ptr(dweight), _stream(dy)))
    return dys, dweight
