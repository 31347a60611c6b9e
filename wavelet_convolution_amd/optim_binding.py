"""Binding of the optimizer's step (argument marshalling only).

The gradients' norm and AdamW over lists of tensors, as defined in wtconv.h.
Every function checks what the plain pointers of the C ABI cannot carry and
calls the C-ABI entry point of the same name on the current stream of the
tensors' device (or on `stream`). There is no fallback.

The states (and fp32 master copies) of a list of tensors stand in one buffer
each, a tensor's from the next multiple of 256 elements on:
`wtconv_adamw_state_count` elements.
"""
from __future__ import annotations

import math

from . import binding as _b
from .block_binding import _elsewhere, _enter

BLOCK = 256


def wtconv_adamw_state_count(params) -> int:
    """Elements of the states' buffers for these tensors (a list; their sizes count only)."""
    return _b.load_native().adamw_state_count(list(params))


def wtconv_adamw_step(params, grads, m, v, step, *, lr, weight_decay, betas=(0.9, 0.999), eps: float = 1e-8,
                      scales=None, master=None, factor=None, lr_factor=None, rng=None, site: int = 0, stream=None):
    """One AdamW step on a list of parameters (fp32 or bf16, all alike), in place, with their gradients (fp32 or
    bf16, all alike; None leaves a parameter and its states as they are).

    m, v: the states, one buffer of wtconv_adamw_state_count(params) elements each, fp32, or float8_e4m3fn with
    `scales` (fp32 [elements / 256, 2]). step: the number of this step (1 for the first), one int64 on the GPU.
    lr, weight_decay: a number, or one for each tensor (a float32 tensor on the host, or a sequence); lr_factor: one
    fp32 number on the GPU that lr is multiplied by. factor: one fp32 number on the GPU that the gradients are
    multiplied by (as wtconv_grad_norm's second result); where it is not finite nothing is changed. master: fp32
    copies of bf16 parameters, laid out as the states. rng (int64 {seed, offset} on the GPU): states in 8 bits are
    rounded stochastically; tensor i uses the generator's site + i, which no dropout or other call with the same rng
    may use at this offset."""
    params, grads = list(params), list(grads)
    if stream is None or not params or not _elsewhere(params[0], stream):
        if _b.load_native().adamw_step(params, grads, m, v, step, lr, weight_decay, *betas, eps, scales, master,
                                       factor, lr_factor, rng, site) is not NotImplemented:
            return
    held = (params, grads, m, v, step, scales, master, factor, lr_factor, rng)
    _enter(wtconv_adamw_step, params[0], stream, held, params, grads, m, v, step, lr=lr, weight_decay=weight_decay,
           betas=betas, eps=eps, scales=scales, master=master, factor=factor, lr_factor=lr_factor, rng=rng, site=site)


def wtconv_adamw_check(params, grads, m, v, step, *, lr, weight_decay, betas=(0.9, 0.999), eps: float = 1e-8,
                       scales=None, master=None, factor=None, lr_factor=None, rng=None, site: int = 0) -> None:
    """Raises what wtconv_adamw_step would raise for these arguments; makes no device call."""
    _b.load_native().adamw_check(list(params), list(grads), m, v, step, lr, weight_decay, *betas, eps, scales, master,
                                 factor, lr_factor, rng, site)


def wtconv_grad_norm(grads, max_norm: float = math.inf, *, step=None, out=None, ws=None, stream=None):
    """A tensor of two fp32 numbers: the norm of all gradients (a list of fp32 and bf16 tensors; None counts nothing)
    and min(1, max_norm / (norm + 1e-6)), NaN where the norm is not finite. step: an int64 on the GPU, increased by
    one where it is finite. ws: a workspace (allocated if None)."""
    grads = list(grads)
    first = next((t for t in grads if t is not None), None)
    if stream is None or first is None or not _elsewhere(first, stream):
        r = _b.load_native().grad_norm(grads, max_norm, step, out, ws)
        if r is not NotImplemented:
            return r
    return _enter(wtconv_grad_norm, first, stream, (grads, step, out, ws), grads, max_norm, step=step, out=out, ws=ws)
