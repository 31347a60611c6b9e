"""Thin ctypes binding of the block operators (argument marshalling only).

Channel norm, block residual and counter dropout, as defined in wtconv.h:
every function takes [B, C, H, W] tensors on the GPU in planar or
channels-last memory order (tokens: H = 1, W tokens, channels last), checks
what the plain pointers of the C ABI cannot carry, and calls the C-ABI entry
point of the same name on the current stream of the tensors' device (or on
`stream`, on which outputs are then allocated too). There is no fallback.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as _b

_DTYPES = {torch.float32: _b.WTCONV_F32, torch.bfloat16: _b.WTCONV_BF16}
_NORMS = {"none": 0, "layer": 1, "rms": 2}
_DROPS = {"none": 0, "element": 1, "sample": 2}
GRADS = ("dx", "dh", "dweight", "dbias", "dgate", "dx_scale")


def _code(table: dict, value, what: str) -> int:
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{what} must be one of {', '.join(map(str, table))}; got {value!r}") from None


def _on_gpu(act, **tensors) -> None:
    """The binding's refusal of host tensors (and of those of another GPU); the quick test first."""
    if isinstance(act, torch.Tensor) and act.is_cuda:
        dev = act.device
        for t in tensors.values():
            if t is not None and not (isinstance(t, torch.Tensor) and t.device == dev):
                break
        else:
            return
    _b._require_gpu(act, **tensors)


def _vector(name: str, t, act) -> None:
    """A parameter of one fp32 number a channel."""
    if t is not None and not (t.dtype is torch.float32 and t.dim() == 1 and t.numel() == act.shape[1]
                              and t.is_contiguous()):
        _b._check_f32(name, t, (act.shape[1],), act)


def _act(name: str, t: torch.Tensor, like: torch.Tensor | None = None) -> tuple[int, int]:
    """(dtype, layout) codes of an activation tensor."""
    if t.dim() != 4 or (like is not None and t.shape != like.shape):
        want = "[B, C, H, W]" if like is None else tuple(like.shape)
        raise ValueError(f"{name} must have shape {want}; got {tuple(t.shape)}")
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be float32 or bfloat16; got {t.dtype}")
    return dt, _b.layout_of(t)


def _rng(rng, act: torch.Tensor) -> None:
    if rng is None or rng.dtype != torch.int64 or rng.numel() != 2 or not rng.is_contiguous():
        raise ValueError(f"a dropout needs rng, a contiguous int64 tensor {{seed, offset}} on {act.device}")


def _gate_code(gate, act: torch.Tensor) -> int:
    if gate is None:
        return 0
    if gate.dim() == 1:
        _vector("gate", gate, act)
        return 1
    _b._check_f32("gate", gate, tuple(act.shape[:2]), act)
    return 2


def _elsewhere(act: torch.Tensor, stream) -> bool:
    """Whether the call has to enter another device or stream first."""
    if stream is None:
        return act.device.index != torch.cuda.current_device()
    if stream.device != act.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {act.device}")
    return stream != torch.cuda.current_stream(act.device)


def _enter(fn, act, stream, tensors, *args, **kw):
    """fn on act's device and on `stream`: outputs and workspace are allocated there, and the tensors that come
    from another stream are marked as in use on it."""
    if stream is None:
        with torch.cuda.device(act.device):
            return fn(*args, **kw)
    for t in tensors:
        for u in t if isinstance(t, (tuple, list)) else (t,):
            if u is not None:
                u.record_stream(stream)
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


def _desc(act, h_code, y_code, norm=0, eps=1e-6, gate=0, drop=0, p=0.0, site=0):
    B, C, H, W = act.shape
    if (B | C | H | W) >> 31:   # the quick test first
        _b._check_i32(B, C, H, W)
    if not 0 <= site < 1 << 31:
        raise ValueError("site must be in 0..2^31-1")
    return _b.WTConvBlockDesc(B, C, H, W, *h_code, *y_code, norm, eps, gate, drop, p, site)


def _empty(shape, dtype, channels_last: bool, device) -> torch.Tensor:
    return torch.empty(shape, dtype=dtype, device=device,
                       memory_format=torch.channels_last if channels_last else torch.contiguous_format)


def _grad(wanted: bool, param, act):
    """A gradient to be written: like its parameter (checked before), or [C] without one."""
    if not wanted:
        return None
    return act.new_empty(act.shape[1], dtype=torch.float32) if param is None else torch.empty_like(param)


# the current stream's handle, without the Stream object around it where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(act) -> int:
    if _raw_stream is None:
        return torch.cuda.current_stream(act.device).cuda_stream
    return _raw_stream(act.device.index)


def _workspace(desc, act, ws):
    """(pointer, bytes) of the workspace, and the tensor that holds it."""
    if ws is not None:
        return _b._ws_ptr(ws), _b._ws_bytes(ws), ws
    n = _b.load_library().wtconv_block_workspace_size(ctypes.byref(desc))
    if n == 0 or n == _NO_SIZE:   # no size: the call itself says what is wrong
        return 0, 0, None
    ws = act.new_empty(n + 256, dtype=torch.uint8)
    return _b._ws_ptr(ws), n, ws


_NO_SIZE = ctypes.c_size_t(-1).value


def _ws_size(desc) -> int:
    n = _b.load_library().wtconv_block_workspace_size(ctypes.byref(desc))
    if n == _NO_SIZE:
        raise _b.WTConvError(2, _b.wtconv_status_string(2))
    return int(n)


def wtconv_block_workspace_size(y, h=None, *, kind: str = "layer", gate=None) -> int:
    """Bytes of workspace of a backward call: of the norm from h's type and memory order into y's (default: the
    same), or of the residual with stream y, block output h and this gate. Makes no device call."""
    h = y if h is None else h
    d = _desc(y, _act("h", h, y), _act("y", y), _code(_NORMS, kind, "kind"), gate=_gate_code(gate, y))
    return _ws_size(d)


def wtconv_block_route(y, h=None, *, kind: str = "layer") -> str:
    """"fused" or "generic": how a norm from h's type and memory order into y's, or the residual with stream y and
    block output h, runs. Makes no device call."""
    h = y if h is None else h
    d = _desc(y, _act("h", h, y), _act("y", y), _code(_NORMS, kind, "kind"))
    r = _b.load_library().wtconv_block_route(ctypes.byref(d))
    if r < 0:
        raise _b.WTConvError(2, _b.wtconv_status_string(2))
    return _b.ROUTES[r]


def wtconv_norm_fwd(x, weight=None, bias=None, *, kind: str = "layer", eps: float = 1e-6, channels_last=None,
                    dtype=None, y=None, stream=None):
    """y = norm(x) * weight + bias over the channels of each pixel. kind: "layer" or "rms"; weight, bias [C] fp32 or
    None. y has x's type and memory order unless `dtype` or `channels_last` (True, False) say otherwise, or `y` is
    given."""
    _on_gpu(x, weight=weight, bias=bias, y=y)
    if _elsewhere(x, stream):
        return _enter(wtconv_norm_fwd, x, stream, (x, weight, bias, y), x, weight, bias, kind=kind, eps=eps,
                      channels_last=channels_last, dtype=dtype, y=y)
    hc = _act("x", x)
    _vector("weight", weight, x)
    _vector("bias", bias, x)
    if y is None:
        same = channels_last is None or bool(channels_last) == (hc[1] == _b.WTCONV_NHWC)
        if same and (dtype is None or dtype == x.dtype):
            y = torch.empty_like(x)
        else:
            y = _empty(x.shape, dtype or x.dtype, hc[1] == _b.WTCONV_NHWC if channels_last is None else channels_last,
                       x.device)
    elif (dtype is not None and y.dtype != dtype) or (
            channels_last is not None and not y.is_contiguous(
                memory_format=torch.channels_last if channels_last else torch.contiguous_format)):
        raise ValueError("y differs from the dtype or memory order asked for")
    d = _desc(x, hc, _act("y", y, x), _code(_NORMS, kind, "kind"), eps)
    _b._check(_b.load_library().wtconv_norm_fwd(ctypes.byref(d), x.data_ptr(), _b._ptr(weight), _b._ptr(bias),
                                                y.data_ptr(), _stream(x)))
    return y


def wtconv_norm_bwd(x, dy, weight=None, bias=None, *, kind: str = "layer", eps: float = 1e-6, want=None, dx=None,
                    ws=None, stream=None):
    """(dx, dweight, dbias) of wtconv_norm_fwd; dx has x's type and memory order. `want`: the names of the
    gradients to compute (default: dx, and those of the parameters given); the others are None. `ws`: a workspace
    of wtconv_block_workspace_size bytes (allocated if None)."""
    _on_gpu(x, dy=dy, weight=weight, bias=bias, dx=dx, ws=ws)
    if _elsewhere(x, stream):
        return _enter(wtconv_norm_bwd, x, stream, (x, dy, weight, bias, dx, ws), x, dy, weight, bias, kind=kind,
                      eps=eps, want=want, dx=dx, ws=ws)
    hc = _act("x", x)
    _vector("weight", weight, x)
    _vector("bias", bias, x)
    wants = (True, weight is not None, bias is not None) if want is None else _wanted(want, ("dx", "dweight", "dbias"))
    d = _desc(x, hc, _act("dy", dy, x), _code(_NORMS, kind, "kind"), eps)
    if not wants[0]:
        dx = None
    elif dx is None:
        dx = torch.empty_like(x)
    elif _act("dx", dx, x) != hc:
        raise ValueError("dx must have x's type and memory order")
    dweight, dbias = _grad(wants[1], weight, x), _grad(wants[2], bias, x)
    wp, wn, ws = _workspace(d, x, ws)
    _b._check(_b.load_library().wtconv_norm_bwd(
        ctypes.byref(d), x.data_ptr(), dy.data_ptr(), _b._ptr(weight), _b._ptr(dx), _b._ptr(dweight), _b._ptr(dbias),
        wp, wn, _stream(x)))
    return dx, dweight, dbias


def _wanted(want, names) -> tuple:
    """For each of the names whether it is wanted."""
    want = tuple(want)
    for n in want:
        if n not in names:
            raise ValueError(f"want names gradients among {', '.join(names)}; got {n!r}")
    return tuple(n in want for n in names)


def _residual_desc(x, h, kind, weight, bias, eps, gate, x_scale, drop, p, rng, site):
    xc, hc = _act("x", x), _act("h", h, x)
    norm, mode = _code(_NORMS, kind, "kind"), _code(_DROPS, drop, "drop")
    if norm == 0 and (weight is not None or bias is not None):
        raise ValueError("weight and bias need a norm (kind)")
    _vector("weight", weight, x)
    _vector("bias", bias, x)
    _vector("x_scale", x_scale, x)
    if mode:
        _rng(rng, x)
    return _desc(x, hc, xc, norm, eps, _gate_code(gate, x), mode, p if mode else 0.0, site)


def wtconv_residual_fwd(x, h, *, kind: str = "none", weight=None, bias=None, eps: float = 1e-6, gate=None,
                        x_scale=None, drop: str = "none", p: float = 0.0, rng=None, site: int = 0, out=None,
                        stream=None):
    """out = x_scale * x + gate * D(norm(h) * weight + bias). x and out share type and memory order, h has its own.
    kind: "none", "layer" or "rms"; gate: [C] or [B, C]; x_scale: [C]; drop: "none", "element" or "sample", with
    probability p from rng (int64 {seed, offset} on the GPU) and site. Parameters are fp32."""
    _on_gpu(x, h=h, weight=weight, bias=bias, gate=gate, x_scale=x_scale, rng=rng, out=out)
    if _elsewhere(x, stream):
        return _enter(wtconv_residual_fwd, x, stream, (x, h, weight, bias, gate, x_scale, rng, out), x, h, kind=kind,
                      weight=weight, bias=bias, eps=eps, gate=gate, x_scale=x_scale, drop=drop, p=p, rng=rng,
                      site=site, out=out)
    d = _residual_desc(x, h, kind, weight, bias, eps, gate, x_scale, drop, p, rng, site)
    if out is None:
        out = torch.empty_like(x)
    elif _act("out", out, x) != (d.y_dtype, d.y_layout):
        raise ValueError("out must have x's type and memory order")
    _b._check(_b.load_library().wtconv_residual_fwd(
        ctypes.byref(d), x.data_ptr(), h.data_ptr(), _b._ptr(weight), _b._ptr(bias), _b._ptr(gate), _b._ptr(x_scale),
        _b._ptr(rng), out.data_ptr(), _stream(x)))
    return out


def wtconv_residual_bwd(dout, h, *, x=None, kind: str = "none", weight=None, bias=None, eps: float = 1e-6, gate=None,
                        x_scale=None, drop: str = "none", p: float = 0.0, rng=None, site: int = 0, want=None,
                        dx=None, dh=None, ws=None, stream=None):
    """(dx, dh, (dweight, dbias, dgate, dx_scale)) of wtconv_residual_fwd. Without an x_scale dx is dout itself
    (unless a dx to write is given); x is needed for dx_scale only. `want`: the names of the gradients to compute
    (default: dx, dh and those of the parameters given); the others are None."""
    _on_gpu(dout, h=h, x=x, weight=weight, bias=bias, gate=gate, x_scale=x_scale, rng=rng, dx=dx, dh=dh, ws=ws)
    if _elsewhere(dout, stream):
        return _enter(wtconv_residual_bwd, dout, stream,
                      (dout, h, x, weight, bias, gate, x_scale, rng, dx, dh, ws), dout, h, x=x, kind=kind,
                      weight=weight, bias=bias, eps=eps, gate=gate, x_scale=x_scale, drop=drop, p=p, rng=rng,
                      site=site, want=want, dx=dx, dh=dh, ws=ws)
    d = _residual_desc(dout, h, kind, weight, bias, eps, gate, x_scale, drop, p, rng, site)
    yc, hc = (d.y_dtype, d.y_layout), (d.h_dtype, d.h_layout)
    if want is None:
        wants = (True, True, weight is not None, bias is not None, gate is not None, x_scale is not None)
    else:
        wants = _wanted(want, GRADS)
        if wants[4] and gate is None:
            raise ValueError("dgate needs a gate")
        if d.norm == 0 and (wants[2] or wants[3]):
            raise ValueError("dweight and dbias need a norm (kind)")
    if wants[5]:
        if x is None:
            raise ValueError("dx_scale needs x")
        if _act("x", x, dout) != yc:
            raise ValueError("x must have dout's type and memory order")
    alias = wants[0] and dx is None and x_scale is None
    if not wants[0]:
        dx = None
    elif dx is not None:
        if _act("dx", dx, dout) != yc:
            raise ValueError("dx must have dout's type and memory order")
    elif not alias:
        dx = torch.empty_like(dout)
    if not wants[1]:
        dh = None
    elif dh is None:
        dh = torch.empty_like(h)
    elif _act("dh", dh, h) != hc:
        raise ValueError("dh must have h's type and memory order")
    dweight, dbias, dgate, dx_scale = (_grad(w, t, dout) for w, t in zip(wants[2:], (weight, bias, gate, x_scale)))
    wp, wn, ws = _workspace(d, dout, ws)
    _b._check(_b.load_library().wtconv_residual_bwd(
        ctypes.byref(d), _b._ptr(x) if dx_scale is not None else 0, h.data_ptr(), dout.data_ptr(), _b._ptr(weight),
        _b._ptr(bias), _b._ptr(gate), _b._ptr(x_scale), _b._ptr(rng), _b._ptr(dx), _b._ptr(dh), _b._ptr(dweight),
        _b._ptr(dbias), _b._ptr(dgate), _b._ptr(dx_scale), wp, wn, _stream(dout)))
    return (dout if alias else dx), dh, (dweight, dbias, dgate, dx_scale)


def wtconv_dropout(x, p: float, rng, *, site: int = 0, mode: str = "element", y=None, stream=None):
    """y = D(x): elements (mode "element") or whole samples b (mode "sample") dropped with probability p by the bits
    of rng (int64 {seed, offset} on the GPU) and site; what is kept is scaled. The mask is never stored: the
    gradient is the same call on dy."""
    _on_gpu(x, rng=rng, y=y)
    if _elsewhere(x, stream):
        return _enter(wtconv_dropout, x, stream, (x, rng, y), x, p, rng, site=site, mode=mode, y=y)
    c = _act("x", x)
    drop = _code(_DROPS, mode, "mode")
    if drop == 0:
        raise ValueError("mode must be element or sample")
    _rng(rng, x)
    if y is None:
        y = torch.empty_like(x)
    elif _act("y", y, x) != c:
        raise ValueError("y must have x's type and memory order")
    d = _desc(x, c, c, drop=drop, p=p, site=site)
    _b._check(_b.load_library().wtconv_dropout(ctypes.byref(d), x.data_ptr(), rng.data_ptr(), y.data_ptr(),
                                               _stream(x)))
    return y
