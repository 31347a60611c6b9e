"""Plain 64-bit form of the block operators on the CPU, with error bounds.

The bounds follow the standard model of fp32 arithmetic: u = 2^-24 a rounded
operation, (n + k) u sum|terms| for a sum of n terms in any order with k more
operations on each. A store rounds by at most half a step of its type:
2^-24 (fp32) or 2^-8 (bf16: eps / 2) relative to the value."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2}
TINY = 2.0 ** -120   # flushed or denormal results


def philox(group, site: int, offset: int, seed: int):
    """Philox4x32-10: [n, 4] uint32 words of the counters (group, site, offset low, offset high)."""
    m = np.uint64(0xFFFFFFFF)
    s32 = np.uint64(32)
    g = np.asarray(group, dtype=np.uint64)
    c = [g, np.full_like(g, site), np.full_like(g, offset & 0xFFFFFFFF), np.full_like(g, (offset >> 32) & 0xFFFFFFFF)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> s32) ^ c[1] ^ np.uint64(k[0]), b & m, (a >> s32) ^ c[3] ^ np.uint64(k[1]), a & m]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, -1).astype(np.uint32)


def keep_mask(shape, mode: str, p: float, seed: int, offset: int, site: int):
    """(mask [B, C, H, W] of truth values, the kept elements' factor)."""
    B, C, H, W = shape
    T = int(np.floor(p * 65536 + 0.5))
    scale = 65536 / (65536 - T) if T < 65536 else 0.0
    if mode == "none" or T == 0:
        return torch.ones(shape, dtype=torch.bool), 1.0
    if mode == "sample":
        w = philox(np.arange(B), site + (1 << 31), offset, seed)[:, 0] & 0xFFFF
        return torch.from_numpy(w >= T).view(B, 1, 1, 1).expand(shape), scale
    G = -(-C // 8)
    w = philox(np.arange(B * H * W * G), site, offset, seed)
    bits = np.stack((w & 0xFFFF, w >> 16), -1).reshape(B, H, W, G * 8)[..., :C]
    return torch.from_numpy(bits >= T).permute(0, 3, 1, 2), scale


def f64(t):
    return None if t is None else t.detach().double().cpu()


def col(v):
    return v.reshape(-1, v.shape[-1], 1, 1)


class Ref:
    """out (or y), and for a dy every gradient, with a bound for each."""

    def __init__(self, h, x=None, kind="none", weight=None, bias=None, eps=1e-6, gate=None, x_scale=None,
                 drop="none", p=0.0, seed=0, offset=0, site=0, dy=None):
        h, x, weight, bias, gate, x_scale, dy = map(f64, (h, x, weight, bias, gate, x_scale, dy))
        B, C, H, W = h.shape
        eps = float(np.float32(eps))   # the descriptor holds it in 32 bits
        mask, k = keep_mask(h.shape, drop, p, seed, offset, site)
        live = mask if drop == "sample" else torch.ones_like(mask)   # a dropped sample's h does not count
        h = torch.where(live, h, torch.zeros_like(h))
        if kind == "none":
            z, r, ez = h, None, torch.zeros_like(h)
        else:
            mean = h.mean(1, keepdim=True) if kind == "layer" else torch.zeros(B, 1, H, W, dtype=h.dtype)
            r = ((h - mean).square().mean(1, keepdim=True) + eps).rsqrt()
            z = (h - mean) * r
            # the mean is off by (C + 2) u max|h|, r by as much of itself again and through the mean's error
            cond = h.abs().amax(1, keepdim=True) * r if kind == "layer" else 0.0
            ez = (C + 16) * U * (cond + z.abs() * (1 + cond))
        w = torch.ones(C, dtype=h.dtype) if weight is None else weight
        v, ev = z * col(w), ez * col(w).abs()
        av = v.abs()
        if bias is not None:
            v, av = v + col(bias), av + col(bias).abs()
        ev = ev + 3 * U * av
        t = torch.where(mask, v * k, torch.zeros_like(v))
        et = torch.where(mask, (ev + U * av) * k, torch.zeros_like(v))
        g = torch.ones(C, dtype=h.dtype) if gate is None else gate
        s = torch.ones(C, dtype=h.dtype) if x_scale is None else x_scale
        out, eo = t * col(g), et * col(g).abs() + 2 * U * (t * col(g)).abs()
        if x is not None:
            out, eo = out + x * col(s), eo + 3 * U * ((x * col(s)).abs() + (t * col(g)).abs())
        self.out, self.out_bound = out, eo
        if dy is None:
            return
        n = B * H * W + 64   # terms of a parameter gradient, and the joining of its partial sums
        rows = (0, 2, 3)
        self.grads, self.bounds = {}, {}

        def put(name, val, bound):
            self.grads[name], self.bounds[name] = val, bound

        def summed(name, a, b, ea, dims, count):
            """sum a b, where a is off by ea"""
            put(name, (a * b).sum(dims), (ea * b.abs()).sum(dims) + count * U * (a * b).abs().sum(dims))

        put("dx", dy * col(s), 2 * U * (dy * col(s)).abs())
        if x is not None:
            summed("dx_scale", x, dy, torch.zeros_like(x), rows, n)
        if gate is not None:
            by_sample = gate.dim() == 2
            summed("dgate", t, dy, et, (2, 3) if by_sample else rows, (H * W + 64) if by_sample else n)
        dv = torch.where(mask, dy * col(g) * k, torch.zeros_like(dy))
        ev = 3 * U * dv.abs()
        if kind == "none":
            put("dh", dv, ev)
            return
        summed("dweight", z, dv, ez + 3 * U * z.abs(), rows, n)
        put("dbias", dv.sum(rows), (n + 3) * U * dv.abs().sum(rows))
        u = dv * col(w)
        m1 = u.mean(1, keepdim=True) if kind == "layer" else 0.0
        m2 = (u * z).mean(1, keepdim=True)
        a1, a2 = u.abs().mean(1, keepdim=True), (u * z).abs().mean(1, keepdim=True)
        dh = r * (u - m1 - z * m2)
        size = r * (u.abs() + a1 + z.abs() * a2)
        # every term is off by (C + 16) u of its size; z's own error enters through z m2 and m2
        bound = (C + 16) * U * 2 * size + r * (ez * m2.abs() + z.abs() * (u.abs() * ez).mean(1, keepdim=True)) \
            + ez.amax(1, keepdim=True) * size   # r's relative error is no larger than that of the largest z
        put("dh", torch.where(live, dh, torch.zeros_like(dh)), bound)


def check(name: str, got, ref, bound):
    """Every element within the bound and the rounding of its type."""
    g = got.detach().double().cpu()
    assert tuple(g.shape) == tuple(ref.shape), (name, tuple(g.shape), tuple(ref.shape))
    if not g.numel():
        return
    allowed = bound + HALF_STEP[got.dtype] * (ref.abs() + bound) + TINY
    off = (g - ref).abs()
    bad = ~(off <= allowed)
    assert not bool(bad.any()), (name, int(bad.sum()), float((off / allowed).max()),
                                 [int(i) for i in bad.nonzero()[0]], float(g[bad][0]), float(ref[bad][0]))
