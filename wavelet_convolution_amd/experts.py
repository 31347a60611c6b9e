"""A block's MLP as a set of experts, but for the matrix products, for PyTorch:
rows sorted by expert, sent there and summed up again, as autograd Functions
over the C-ABI entry points.

    route = expert_sort(expert, E)            expert [B, H, W, K] (or [N, K]): K of E experts for each row
    xs = expert_rows(rows, route)             rows [B, H, W, C] -> [B H W K, C], an expert's rows together
    ys = (grouped products of xs, with route.offsets[1:] as the groups' ends)
    y  = expert_sum(ys, weight, route)        weight [B, H, W, K] fp32 -> [B, H, W, C]

A number outside 0..E-1 is no expert (padding, or a row over an expert's
capacity): its rows of xs come last and are zeros, and it adds nothing to y.
Rows are fp32 or bf16. Every step of the computation runs in libwtconv.so.
Tensors must be on the GPU: there is no CPU path. A second derivative raises
an error.
"""
from __future__ import annotations

from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import expert_binding as _eb
from .block import _gpu, _names


class ExpertRoute(NamedTuple):
    """order [N K]: the slots (row * K + k) sorted by expert; place [..., K]: each slot's place in it; offsets
    [E + 1]: expert e's places are offsets[e] .. offsets[e + 1] - 1, and offsets[E] of them have an expert."""
    order: torch.Tensor
    place: torch.Tensor
    offsets: torch.Tensor


def expert_sort(expert: torch.Tensor, experts: int) -> ExpertRoute:
    """The routing of slots with these experts (int32 or int64 [..., K])."""
    _gpu(expert)
    return ExpertRoute(*_eb.wtconv_expert_sort(expert.contiguous(), experts))


class ExpertRowsFunction(torch.autograd.Function):
    """xs[place[n, k]] = x[n]."""

    @staticmethod
    def forward(ctx, x, place, offsets):
        _gpu(x, place, offsets)
        ctx.save_for_backward(place, offsets)
        return _eb.wtconv_expert_rows_fwd(x.contiguous(), place, offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs):
        place, offsets = ctx.saved_tensors
        return _eb.wtconv_expert_rows_bwd(dxs.contiguous(), place, offsets), None, None


class ExpertSumFunction(torch.autograd.Function):
    """y[n] = sum_k weight[n, k] ys[place[n, k]]."""

    @staticmethod
    def forward(ctx, ys, weight, place, offsets):
        _gpu(ys, weight, place, offsets)
        ys, weight = ys.contiguous(), weight.contiguous()
        ctx.save_for_backward(ys, weight, place, offsets)
        return _eb.wtconv_expert_sum_fwd(ys, weight, place, offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        ys, weight, place, offsets = ctx.saved_tensors
        want = _names(ctx, ((0, "dys"), (1, "dweight")))
        return *_eb.wtconv_expert_sum_bwd(dy.contiguous(), ys, weight, place, offsets, want=want), None, None


def expert_rows(x: torch.Tensor, route: ExpertRoute) -> torch.Tensor:
    """The rows of x [..., C] at their slots' places, [N K, C] (differentiable)."""
    return ExpertRowsFunction.apply(x, route.place, route.offsets)


def expert_sum(ys: torch.Tensor, weight: torch.Tensor, route: ExpertRoute) -> torch.Tensor:
    """The weighted sum of each row's slots' rows of ys [N K, C], [..., C] (differentiable in ys and weight)."""
    return ExpertSumFunction.apply(ys, weight, route.place, route.offsets)
