"""The rest of a WTConv block that is not a matrix product, for PyTorch:
channel norm, block residual and counter dropout as autograd Functions and
nn.Modules over the C-ABI entry points.

    u   = norm(mixer(x))                  ChannelNorm2d: planar in, channels-last rows out
    h   = linear(drop(gelu(linear(u))))   CounterDropout on the hidden rows
    out = s * x + g * D(norm(h))          BlockResidual2d: channels-last h added to a planar x

Tensors are [B, C, H, W] in planar or channels-last memory order (a linear
layer's [B, H, W, C] rows are ``rows.permute(0, 3, 1, 2)``; tokens [B, S, C]
are H = 1, W = S), fp32 or bf16; parameters are fp32. The backward passes keep
inputs only (the residual's h always, its x for the gradient of an x_scale):
row statistics and dropout masks are computed again. Every step of the
computation runs in libwtconv.so. Tensors must be on the GPU: there is no CPU
path. A second derivative raises an error.

Dropout reads its seed and offset from a tensor on the GPU (`dropout_rng`).
One tensor serves a whole model, each use with a site number of its own; the
caller changes the offset once per step, after the backward pass:
``rng[1] += 1`` (autograd raises an error where it was changed in between).
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding as _b
from . import block_binding as _bb


def dropout_rng(seed: int, device="cuda") -> torch.Tensor:
    """{seed, offset = 0} for the dropout operators."""
    return torch.tensor([seed, 0], dtype=torch.int64, device=device)


def _gpu(*ts) -> None:
    for t in ts:
        if t is not None and not t.is_cuda:
            raise RuntimeError("the block operators run on the GPU only (libwtconv.so); got a tensor on "
                               f"{t.device} - there is no CPU implementation")


def _is_dense(t: torch.Tensor) -> bool:
    """Whether t is planar or channels last."""
    return t.is_contiguous() or (t.dim() == 4 and t.is_contiguous(memory_format=torch.channels_last))


def _dense(t: torch.Tensor, like: torch.Tensor | None = None) -> torch.Tensor:
    """t itself where it is planar or channels last, else a copy in the memory order of `like`."""
    if _is_dense(t):
        return t
    cl = like is not None and _b.layout_of(like) == _b.WTCONV_NHWC
    return t.contiguous(memory_format=torch.channels_last if cl else torch.contiguous_format)


def _names(ctx, pairs) -> tuple:
    return tuple(n for i, n in pairs if ctx.needs_input_grad[i])


class ChannelNormFunction(torch.autograd.Function):
    """y = norm(x) * weight + bias over the channels of each pixel."""

    @staticmethod
    def forward(ctx, x, weight, bias, kind, eps, channels_last, dtype):
        _gpu(x, weight, bias)
        x = _dense(x)
        ctx.save_for_backward(x, weight, bias)
        ctx.opts = dict(kind=kind, eps=eps)
        return _bb.wtconv_norm_fwd(x, weight, bias, channels_last=channels_last, dtype=dtype, **ctx.opts)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, bias = ctx.saved_tensors
        want = _names(ctx, ((0, "dx"), (1, "dweight"), (2, "dbias")))
        grads = _bb.wtconv_norm_bwd(x, _dense(dy, x), weight, bias, want=want, **ctx.opts)
        return *grads, None, None, None, None


class BlockResidualFunction(torch.autograd.Function):
    """out = x_scale * x + gate * D(norm(h) * weight + bias)."""

    @staticmethod
    def forward(ctx, x, h, weight, bias, gate, x_scale, rng, kind, eps, drop, p, site):
        _gpu(x, h, weight, bias, gate, x_scale, rng)
        x, h = _dense(x), _dense(h, x)
        ctx.opts = dict(kind=kind, eps=eps, drop=drop, p=p, site=site)
        # x is read again for the gradient of its scale only
        ctx.save_for_backward(x if x_scale is not None else None, h, weight, bias, gate, x_scale, rng)
        ctx.order = torch.channels_last if _b.layout_of(x) == _b.WTCONV_NHWC else torch.contiguous_format
        return _bb.wtconv_residual_fwd(x, h, weight=weight, bias=bias, gate=gate, x_scale=x_scale, rng=rng,
                                       **ctx.opts)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        x, h, weight, bias, gate, x_scale, rng = ctx.saved_tensors
        if x is not None or not _is_dense(dout):
            dout = dout.contiguous(memory_format=ctx.order)   # as x, which is read beside it
        want = _names(ctx, ((0, "dx"), (1, "dh"), (2, "dweight"), (3, "dbias"), (4, "dgate"), (5, "dx_scale")))
        if not want:
            return (None,) * 12
        dx, dh, (dweight, dbias, dgate, dx_scale) = _bb.wtconv_residual_bwd(
            dout, h, x=x, weight=weight, bias=bias, gate=gate, x_scale=x_scale, rng=rng, want=want, **ctx.opts)
        return dx, dh, dweight, dbias, dgate, dx_scale, None, None, None, None, None, None


class CounterDropoutFunction(torch.autograd.Function):
    """y = D(x); the gradient makes the same mask again."""

    @staticmethod
    def forward(ctx, x, rng, p, site, mode):
        _gpu(x, rng)
        ctx.save_for_backward(rng)
        ctx.opts = dict(site=site, mode=mode)
        ctx.p = p
        return _bb.wtconv_dropout(_dense(x), p, rng, **ctx.opts)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        rng, = ctx.saved_tensors
        return _bb.wtconv_dropout(_dense(dy), ctx.p, rng, **ctx.opts), None, None, None, None


def channel_norm(x, weight=None, bias=None, kind: str = "layer", eps: float = 1e-6, channels_last=None, dtype=None):
    """Functional channel norm (differentiable): LayerNorm ("layer") or RMSNorm ("rms") over dim 1 of [B, C, H, W],
    into x's memory order or the one that `channels_last` names, in x's type or `dtype`."""
    return ChannelNormFunction.apply(x, weight, bias, kind, eps, channels_last, dtype)


def block_residual(x, h, *, kind: str = "none", weight=None, bias=None, eps: float = 1e-6, gate=None, x_scale=None,
                   drop: str = "none", p: float = 0.0, rng=None, site: int = 0):
    """Functional block residual (differentiable): x_scale * x + gate * D(norm(h) * weight + bias), in x's type and
    memory order."""
    return BlockResidualFunction.apply(x, h, weight, bias, gate, x_scale, rng if drop != "none" else None, kind, eps,
                                       drop, p, site)


def counter_dropout(x, p: float, rng, site: int = 0, mode: str = "element"):
    """Functional counter dropout (differentiable) of elements, or of whole samples (mode "sample")."""
    return CounterDropoutFunction.apply(x, rng, p, site, mode)


def _check_p(p: float) -> float:
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"a dropout probability lies in 0..1; got {p}")
    return float(p)


class ChannelNorm2d(torch.nn.Module):
    """LayerNorm or RMSNorm over the channels of each pixel. Parameters
    (fp32): ``weight`` [C] (ones) and, unless bias=False, ``bias`` [C]
    (zeros); neither with affine=False. channels_last=True writes the rows
    that a linear layer takes (``y.permute(0, 2, 3, 1)`` is contiguous)
    whatever the input's memory order; None keeps that order."""

    def __init__(self, channels: int, kind: str = "layer", eps: float = 1e-6, affine: bool = True, bias: bool = True,
                 channels_last=None, device=None):
        super().__init__()
        if channels < 1 or kind not in ("layer", "rms") or not eps > 0:
            raise ValueError("channels >= 1, kind 'layer' or 'rms' and eps > 0 are required")
        self.channels, self.kind, self.eps, self.channels_last = channels, kind, eps, channels_last
        f32 = dict(dtype=torch.float32, device=device)
        self.weight = torch.nn.Parameter(torch.ones(channels, **f32)) if affine else None
        self.bias = torch.nn.Parameter(torch.zeros(channels, **f32)) if affine and bias else None

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.dim() != 4 or x.shape[1] != self.channels:
            raise ValueError(f"expected [B, {self.channels}, H, W], got {tuple(x.shape)}")
        return channel_norm(x, self.weight, self.bias, self.kind, self.eps, self.channels_last)

    def extra_repr(self) -> str:
        return (f"channels={self.channels}, kind={self.kind!r}, eps={self.eps}, "
                f"affine={self.weight is not None}, channels_last={self.channels_last}")


class BlockResidual2d(torch.nn.Module):
    """The end of a block: out = x_scale * x + gate * D(norm(h)).

    norm: "none", "layer" or "rms" (with ``weight`` and ``bias`` [C]);
    layer_scale: initial value of a learned per-channel gate ``gate`` [C], or
    None for no such gate (a gate per sample [B, C] may then be passed to
    forward); x_scale=True: a learned per-channel factor ``x_scale`` [C] on
    the stream (ones); drop "element" or "sample" with probability p, active
    in training mode, from the rng given to forward and this use's site."""

    def __init__(self, channels: int, norm: str = "none", eps: float = 1e-6, bias: bool = True, layer_scale=1e-6,
                 x_scale: bool = False, drop: str = "none", p: float = 0.0, site: int = 0, device=None):
        super().__init__()
        if channels < 1 or norm not in ("none", "layer", "rms") or not eps > 0 \
                or drop not in ("none", "element", "sample"):
            raise ValueError("channels >= 1, norm 'none', 'layer' or 'rms', eps > 0 and drop 'none', 'element' or "
                             "'sample' are required")
        self.channels, self.norm, self.eps = channels, norm, eps
        self.drop, self.p, self.site = drop, _check_p(p), site
        f32 = dict(dtype=torch.float32, device=device)
        self.weight = torch.nn.Parameter(torch.ones(channels, **f32)) if norm != "none" else None
        self.bias = torch.nn.Parameter(torch.zeros(channels, **f32)) if norm != "none" and bias else None
        self.gate = None if layer_scale is None else torch.nn.Parameter(torch.full((channels,), float(layer_scale),
                                                                                   **f32))
        self.x_scale = torch.nn.Parameter(torch.ones(channels, **f32)) if x_scale else None

    def forward(self, x: torch.Tensor, h: torch.Tensor, rng=None, gate=None) -> torch.Tensor:
        if x.dim() != 4 or x.shape[1] != self.channels:
            raise ValueError(f"expected [B, {self.channels}, H, W], got {tuple(x.shape)}")
        if gate is not None and self.gate is not None:
            raise ValueError("this residual has a layer scale: no other gate can be passed")
        return block_residual(x, h, kind=self.norm, weight=self.weight, bias=self.bias, eps=self.eps,
                              gate=self.gate if gate is None else gate, x_scale=self.x_scale,
                              drop=self.drop if self.training and self.p > 0 else "none", p=self.p, rng=rng,
                              site=self.site)

    def extra_repr(self) -> str:
        return (f"channels={self.channels}, norm={self.norm!r}, layer_scale={self.gate is not None}, "
                f"x_scale={self.x_scale is not None}, drop={self.drop!r}, p={self.p}, site={self.site}")


class CounterDropout(torch.nn.Module):
    """Dropout of elements (or of whole samples) whose mask is a function of
    (rng, site, element) and is never stored; the identity in eval mode."""

    def __init__(self, p: float, site: int, mode: str = "element"):
        super().__init__()
        if mode not in ("element", "sample"):
            raise ValueError("mode must be 'element' or 'sample'")
        self.p, self.site, self.mode = _check_p(p), site, mode

    def forward(self, x: torch.Tensor, rng: torch.Tensor) -> torch.Tensor:
        if not self.training or self.p == 0:
            return x
        return counter_dropout(x, self.p, rng, self.site, self.mode)

    def extra_repr(self) -> str:
        return f"p={self.p}, site={self.site}, mode={self.mode!r}"
