"""Thin ctypes binding of the optimizer's step (argument marshalling only).

The gradients' norm and AdamW over lists of tensors, as defined in wtconv.h.
Every function checks what the plain pointers of the C ABI cannot carry and
calls the C-ABI entry point of the same name on the current stream of the
tensors' device (or on `stream`). There is no fallback.

The states (and fp32 master copies) of a list of tensors stand in one buffer
each, a tensor's from the next multiple of 256 elements on:
`wtconv_adamw_state_count` elements.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import binding as _b
from .block_binding import _DTYPES, _elsewhere, _enter, _stream

BLOCK = 256

_numel, _data_ptr = torch.Tensor.numel, torch.Tensor.data_ptr
_contiguous, _same_size = torch.Tensor.is_contiguous, torch.Tensor.is_same_size


def _list(name: str, ts) -> list:
    ts = list(ts)
    for t in ts:
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be tensors; got {type(t).__name__}")
    return ts


def _all_on_gpu(dev, **lists) -> None:
    """Every tensor on the same GPU: a host pointer in a kernel's argument is a memory fault."""
    if dev.type != "cuda":
        raise ValueError(f"the optimizer's step takes GPU tensors, got one on {dev}")
    for name, ts in lists.items():
        for d in {t.device for t in ts if t is not None}:
            if d != dev:
                raise ValueError(f"{name} must be on {dev}, as the others; got one on {d}")


def _dense(name: str, ts) -> None:
    if not all(map(_contiguous, ts)):
        raise ValueError(f"{name} must be contiguous tensors")


def _i64(values):
    return (ctypes.c_int64 * len(values))(*values)


def _pointers(ts):
    return (ctypes.c_void_p * len(ts))(*[0 if t is None else t.data_ptr() for t in ts])


def wtconv_adamw_state_count(params) -> int:
    """Elements of the states' buffers for these tensors (a list; their sizes count only)."""
    counts = _i64(list(map(_numel, params)))
    n = _b.load_library().wtconv_adamw_state_count(counts, len(counts))
    if n < 0:
        raise _b.WTConvError(2, _b.wtconv_status_string(2))
    return n


def _buffer(name: str, t, dtype, n: int) -> None:
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements; got {tuple(t.shape)} {t.dtype}")


def _scalar(name: str, t, dtype) -> None:
    if t is not None and (t.dtype is not dtype or t.numel() != 1):
        raise ValueError(f"{name} must be a tensor of one {dtype} number; got {tuple(t.shape)} {t.dtype}")


def _each(name: str, value, n: int):
    """n fp32 numbers on the host: one number for all, or a sequence or CPU tensor of them."""
    if isinstance(value, torch.Tensor):
        if value.device.type != "cpu" or value.numel() != n:
            raise ValueError(f"{name} must be a number, or {n} on the host; got {tuple(value.shape)} on {value.device}")
        value = value.tolist() if value.dtype is not torch.float32 or not value.is_contiguous() else value
    if isinstance(value, torch.Tensor):
        return value.data_ptr(), value
    if isinstance(value, (int, float)):
        a = (ctypes.c_float * n)(*[value] * n)
    else:
        value = list(value)
        if len(value) != n:
            raise ValueError(f"{name} must be a number, or one for each of the {n} tensors; got {len(value)}")
        a = (ctypes.c_float * n)(*value)
    return ctypes.addressof(a), a


def wtconv_adamw_step(params, grads, m, v, step, *, lr, weight_decay, betas=(0.9, 0.999), eps: float = 1e-8,
                      scales=None, master=None, factor=None, lr_factor=None, rng=None, site: int = 0, stream=None):
    """One AdamW step on a list of parameters (fp32 or bf16, all alike), in place, with their gradients (fp32 or
    bf16, all alike; None leaves a parameter and its states as they are).

    m, v: the states, one buffer of wtconv_adamw_state_count(params) elements each, fp32, or float8_e4m3fn with
    `scales` (fp32 [elements / 256, 2]). step: the number of this step (1 for the first), one int64 on the GPU.
    lr, weight_decay: a number, or one for each tensor (on the host); lr_factor: one fp32 number on the GPU that lr is
    multiplied by. factor: one fp32 number on the GPU that the gradients are multiplied by (as wtconv_grad_norm's
    second result); where it is not finite nothing is changed. master: fp32 copies of bf16 parameters, laid out as the
    states. rng (int64 {seed, offset} on the GPU): states in 8 bits are rounded stochastically; tensor i uses the
    generator's site + i."""
    params, grads = _list("params", params), list(grads)
    if len(params) != len(grads) or not params:
        raise ValueError(f"one gradient (or None) a parameter, and one at least, are required; got {len(params)} and "
                         f"{len(grads)}")
    some = _list("grads", [g for g in grads if g is not None])
    dev = params[0].device
    single = [t for t in (m, v, step, scales, master, factor, lr_factor, rng) if t is not None]
    _all_on_gpu(dev, params=params, grads=some, **{"the states and numbers": _list("states", single)})
    if _elsewhere(params[0], stream):
        return _enter(wtconv_adamw_step, params[0], stream, (params, grads, single), params, grads, m, v, step, lr=lr,
                      weight_decay=weight_decay, betas=betas, eps=eps, scales=scales, master=master, factor=factor,
                      lr_factor=lr_factor, rng=rng, site=site)
    types, gtypes = {t.dtype for t in params}, {t.dtype for t in some} or {torch.float32}
    if len(types) != 1 or len(gtypes) != 1 or not (types | gtypes) <= _DTYPES.keys():
        raise ValueError("parameters must be all float32 or all bfloat16, and so must gradients; got "
                         f"{', '.join(map(str, types))} and {', '.join(map(str, gtypes))}")
    _dense("params", params)
    _dense("grads", some)
    if len(some) == len(params):
        alike = all(map(_same_size, params, grads))
    else:
        alike = all(g is None or p.is_same_size(g) for p, g in zip(params, grads))
    if not alike:
        raise ValueError("gradients must have their parameters' shapes")
    counts = _i64(list(map(_numel, params)))
    n, lib = len(params), _b.load_library()
    all_ = lib.wtconv_adamw_state_count(counts, n)
    if all_ < 0:
        raise _b.WTConvError(2, _b.wtconv_status_string(2))
    state = torch.float32 if scales is None else torch.float8_e4m3fn
    _buffer("m", m, state, all_)
    _buffer("v", v, state, all_)
    if scales is not None:
        _buffer("scales", scales, torch.float32, all_ // BLOCK * 2)
    if master is not None:
        if types != {torch.bfloat16}:
            raise ValueError("master copies are for bfloat16 parameters")
        _buffer("master", master, torch.float32, all_)
    if step is None:
        raise ValueError("step, one int64 number on the GPU, is required")
    _scalar("step", step, torch.int64)
    _scalar("factor", factor, torch.float32)
    _scalar("lr_factor", lr_factor, torch.float32)
    if rng is not None and (rng.dtype is not torch.int64 or rng.numel() != 2 or not rng.is_contiguous()
                            or scales is None):
        raise ValueError("rng must be a contiguous int64 tensor {seed, offset}, for states in 8 bits")
    if not 0 <= site < 1 << 31:
        raise ValueError("site must be in 0..2^31-1")
    lr_ptr, lr_held = _each("lr", lr, n)
    wd_ptr, wd_held = _each("weight_decay", weight_decay, n)
    d = _b.WTConvAdamWDesc(_DTYPES[types.pop()], _DTYPES[gtypes.pop()], 32 if scales is None else 8, site, *betas, eps)
    _b._check(lib.wtconv_adamw_step(
        ctypes.byref(d), n, _pointers(params), _pointers(grads), counts, lr_ptr, wd_ptr, m.data_ptr(), v.data_ptr(),
        _b._ptr(scales), _b._ptr(master), step.data_ptr(), _b._ptr(factor), _b._ptr(lr_factor), _b._ptr(rng),
        _stream(params[0])))
    del lr_held, wd_held
    # autograd's own record of changes in place, as torch's operations keep it
    torch.autograd.graph.increment_version(params)


def wtconv_grad_norm(grads, max_norm: float = math.inf, *, step=None, out=None, ws=None, stream=None):
    """A tensor of two fp32 numbers: the norm of all gradients (a list of fp32 and bf16 tensors; None counts nothing)
    and min(1, max_norm / (norm + 1e-6)), NaN where the norm is not finite. step: an int64 on the GPU, increased by
    one where it is finite. ws: a workspace (allocated if None)."""
    grads = _list("grads", [g for g in grads if g is not None])
    if not grads:
        raise ValueError("at least one gradient is required")
    dev = grads[0].device
    single = [t for t in (step, out, ws) if t is not None]
    _all_on_gpu(dev, grads=grads, **{"step, out and ws": _list("step, out and ws", single)})
    if _elsewhere(grads[0], stream):
        return _enter(wtconv_grad_norm, grads[0], stream, (grads, single), grads, max_norm, step=step, out=out, ws=ws)
    types = [_DTYPES.get(t.dtype) for t in grads]
    if None in types:
        raise ValueError("gradients must be float32 or bfloat16")
    if not max_norm > 0:
        raise ValueError(f"max_norm must be above 0 (infinity: no clipping); got {max_norm}")
    _dense("grads", grads)
    _scalar("step", step, torch.int64)
    if out is None:
        out = torch.empty(2, dtype=torch.float32, device=dev)
    else:
        _buffer("out", out, torch.float32, 2)
    n, lib = len(grads), _b.load_library()
    if ws is None:
        ws = torch.empty(lib.wtconv_grad_norm_workspace_size(n) + 256, dtype=torch.uint8, device=dev)
    _b._check(lib.wtconv_grad_norm(n, _pointers(grads), _i64(list(map(_numel, grads))), (ctypes.c_int32 * n)(*types),
                                   max_norm, _b._ptr(step), out.data_ptr(), _b._ws_ptr(ws), _b._ws_bytes(ws),
                                   _stream(grads[0])))
    return out
