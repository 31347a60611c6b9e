"""AdamW for PyTorch over the C-ABI entry points: every parameter of a group in
one call, states in 32 or in 8 bits, the gradients' clipping and the step's
number on the GPU.

    optim = AdamW(model.parameters(), lr=1e-3, weight_decay=0.05, state_bits=8, max_norm=1.0)
    loss.backward()
    optim.step()

The update is that of torch.optim.AdamW with the bias corrections of one step
count for all parameters. Parameters are contiguous, fp32, or bf16 with fp32
master copies (master=False: without). Tensors must be on the GPU: there is no
CPU path.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import optim_binding as _ob


class AdamW(torch.optim.Optimizer):
    """Parameter groups may set lr, betas, eps, weight_decay and state_bits of
    their own.

    state_bits: 32 or 8 (a block of 256 elements shares a scale; the first
    moment and the second one's root are e4m3 numbers). rng: an int64
    {seed, offset} on the GPU (`dropout_rng`), for stochastic rounding of 8-bit
    states; parameter i (counted over all groups) uses the generator's site
    `site + i`, and the caller changes the offset once per step. No other use
    of the same rng, dropouts among them, may have one of these sites: its bits
    would be the same (the default is far above a model's dropouts; another
    optimizer with this rng needs a site of its own). max_norm:
    gradients are scaled down to this norm over all of them, and a step whose
    gradients are not finite changes nothing and is not counted (inf: no
    clipping, but such steps are skipped; None: neither, and no norm is
    computed). `last_norm` is the last step's {norm, factor} on the GPU.

    The states of a group's parameters stand in one buffer each. A parameter
    without a gradient is left as it is in that step, and a step that raises an
    error for its arguments changes nothing in any group. step() makes no copy to
    the host and waits for nothing, so it can be captured into a graph after a
    first step (a graph keeps lr and the other numbers of its capture, but for
    `lr_factor`, an optional fp32 number on the GPU that lr is multiplied by).
    A group's states are made at its first step, master copies from the
    parameters as they are then: call `renew_master` after changing bf16
    parameters in another way, or the next step goes on from the copies."""

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 1e-2,
                 state_bits: int = 32, master: bool = True, max_norm=None, rng=None, site: int = 1 << 30, lr_factor=None):
        if max_norm is not None and not max_norm > 0:
            raise ValueError(f"max_norm must be above 0, or None; got {max_norm}")
        self.master, self.max_norm = master, max_norm
        self.rng, self.site, self.lr_factor = rng, site, lr_factor
        self.last_norm = self._step = None
        self._buffers = []   # of each group: None, or a dict of its states
        betas = tuple(betas) if hasattr(betas, "__iter__") else betas
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, state_bits=state_bits))
        if rng is not None and all(g["state_bits"] != 8 for g in self.param_groups):
            raise ValueError("rng is for states in 8 bits")

    def __getstate__(self):
        own = ("master", "max_norm", "rng", "site", "lr_factor", "last_norm", "_step", "_buffers")
        return {**super().__getstate__(), **{k: self.__dict__[k] for k in own}}

    def add_param_group(self, group):
        if self._step is not None:
            raise RuntimeError("parameter groups are added before the first step: all share its count")
        super().add_param_group(group)
        g, params = self.param_groups[-1], self._params()
        why = None
        if any(p.dtype not in (torch.float32, torch.bfloat16) or p.dtype != g["params"][0].dtype for p in g["params"]):
            why = "the parameters of a group must be all float32 or all bfloat16"
        elif any(p.device != params[0].device for p in g["params"]):
            why = "all parameters must be on one device"
        elif any(not p.is_contiguous() for p in g["params"]):
            why = "parameters must be contiguous (the states have their elements' order)"
        else:
            why = _wrong_numbers(g)
        if why:
            self.param_groups.pop()
            raise ValueError(why)
        self._buffers.append(None)

    def _params(self) -> list:
        return [p for g in self.param_groups for p in g["params"]]

    def _shapes(self) -> list:
        return [[tuple(p.shape) for p in g["params"]] for g in self.param_groups]

    def _make(self, group) -> dict:
        params, eight = group["params"], group["state_bits"] == 8
        if not params:
            return {}
        n, dev = _ob.wtconv_adamw_state_count(params), params[0].device
        kind = torch.float8_e4m3fn if eight else torch.float32
        b = {"m": torch.zeros(n, dtype=kind, device=dev), "v": torch.zeros(n, dtype=kind, device=dev)}
        if eight:
            b["scales"] = torch.zeros(n // _ob.BLOCK, 2, device=dev)
        if self.master and params[0].dtype == torch.bfloat16:
            b["master"] = torch.zeros(n, device=dev)
            _copy(params, b["master"])
        return b

    @torch.no_grad()
    def renew_master(self) -> None:
        """The master copies made again from the parameters."""
        for g, b in zip(self.param_groups, self._buffers):
            if b and "master" in b:
                _copy(g["params"], b["master"])

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        groups, grads = [], []
        for g in self.param_groups:
            ts = [_dense(p.grad) for p in g["params"]]
            there = [t for t in ts if t is not None]
            groups.append((g, ts, there))
            grads += there
        if not grads:
            return loss
        step, buffers = self._step, self._buffers
        if step is None or None in buffers:
            if grads[0].is_cuda and torch.cuda.is_current_stream_capturing():
                raise RuntimeError("the first step makes the states, which a graph would make again at every replay: "
                                   "take a step before the capture")
            buffers = [self._make(g) if b is None else b for g, b in zip(self.param_groups, buffers)]
            if step is None:
                step = torch.zeros(1, dtype=torch.int64, device=grads[0].device)
        calls, site = [], self.site
        for (g, ts, there), b in zip(groups, buffers):
            if there:
                calls.append(((g["params"], ts), dict(
                    step=step, lr=_number("lr", g["lr"]), weight_decay=_number("weight_decay", g["weight_decay"]),
                    betas=g["betas"], eps=g["eps"], lr_factor=self.lr_factor,
                    rng=self.rng if g["state_bits"] == 8 else None, site=site, **b)))
            site += len(ts)
        # a step that is refused leaves the count, the states and every group as they were
        for lists, kw in calls:
            _ob.wtconv_adamw_check(*lists, **kw)
        if self.max_norm is None:
            step += 1
            factor = None
        else:
            self.last_norm = _ob.wtconv_grad_norm(grads, self.max_norm, step=step)
            factor = self.last_norm[1:]
        self._step, self._buffers = step, buffers
        for lists, kw in calls:
            _ob.wtconv_adamw_step(*lists, factor=factor, **kw)
        return loss

    def state_dict(self) -> dict:
        """{"state": {"step", "buffers", "shapes"}, "param_groups"}: the states' buffers as they are (a group's are
        None before its first step), not a state for each parameter, and the parameters' shapes, which say whose."""
        groups = super().state_dict()["param_groups"]
        return {"state": {"step": self._step, "buffers": [b and dict(b) for b in self._buffers],
                          "shapes": self._shapes()},
                "param_groups": groups}

    @torch.no_grad()
    def load_state_dict(self, state_dict) -> None:
        """States are copied into the buffers that are there, so that a captured step goes on with them."""
        state, groups = state_dict["state"], state_dict["param_groups"]
        if len(groups) != len(self.param_groups) or any(
                len(a["params"]) != len(b["params"]) for a, b in zip(groups, self.param_groups)):
            raise ValueError("the state has other parameter groups than this optimizer")
        new = []
        shapes = self._shapes()
        # the sums of two lists of shapes may agree (states saved without shapes: as they come)
        for b, g, own, here, there in zip(state["buffers"], self.param_groups, self._buffers, shapes,
                                          state.get("shapes", shapes)):
            if b is not None and here != [tuple(s) for s in there]:
                raise ValueError("the state is of other parameters: their shapes differ, or their order")
            like = None if b is None else own or self._make(g)
            if like is not None and (like.keys() != b.keys() or any(
                    like[k].shape != t.shape or like[k].dtype != t.dtype for k, t in b.items())):
                raise ValueError("the state is of other parameters, or of other state_bits or master copies")
            new.append(like)
        for like, b in zip(new, state["buffers"]):
            for k in like or ():
                like[k].copy_(b[k])
        self._buffers = new
        if state["step"] is None or self._step is None:
            self._step = None if state["step"] is None else state["step"].to(self._params()[0].device, copy=True)
        else:
            self._step.copy_(state["step"])
        for mine, other in zip(self.param_groups, groups):
            mine.update({k: v for k, v in other.items() if k != "params"})


def _number(name: str, v):
    """A number on the host; several of them (one for each parameter) as they are."""
    if type(v) is float:
        return v
    if isinstance(v, torch.Tensor):
        if v.device.type != "cpu":
            raise ValueError(f"{name} must be a number on the host (lr_factor scales rates on the GPU)")
        return float(v) if v.numel() == 1 else v
    return v if isinstance(v, (list, tuple)) else float(v)


def _wrong_numbers(g):
    """What is wrong with a group's numbers, as the step sees them (in fp32), or None."""
    def f32(name):
        return ctypes.c_float(_number(name, g[name])).value

    try:
        betas = [float(b) for b in g["betas"]]
        ok = (0 <= f32("lr") < math.inf and 0 <= f32("weight_decay") < math.inf
              and torch.finfo(torch.float32).tiny <= f32("eps") < math.inf
              and len(betas) == 2 and all(0 <= b < 1 for b in betas) and g["state_bits"] in (8, 32))
    except (TypeError, ValueError, RuntimeError) as e:
        return f"a group's numbers: {e}"
    return None if ok else ("lr >= 0, weight_decay >= 0, eps of 2^-126 at least, two betas in [0, 1) and state_bits "
                            "8 or 32 are required")


def _dense(grad):
    return grad if grad is None or grad.is_contiguous() else grad.contiguous()


def _copy(params, master) -> None:
    """fp32 copies of the parameters, each at its place in the states' layout."""
    at = 0
    for p in params:
        master[at:at + p.numel()].copy_(p.detach().reshape(-1))
        at += -(-p.numel() // _ob.BLOCK) * _ob.BLOCK
