"""Block operators: channel norm, block residual, counter dropout.

CPU: the generator's published test vectors, argument checks of the C-ABI and
the binding, module construction. GPU: forward and every gradient against the
plain 64-bit form of tests/_block_ref.py, at sizes, types, memory orders and
masks where they can go wrong, with bounds from the arithmetic."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

from tests._block_ref import Ref, check, keep_mask, philox
from wavelet_convolution_amd import binding as wt
from wavelet_convolution_amd import block as blk
from wavelet_convolution_amd import block_binding as bb

gpu = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]


def on_gpu(fn):
    for m in gpu:
        fn = m(fn)
    return fn


# ------------------------------------------------------------------- CPU

def test_generator_reference_vectors():
    """The test generator reproduces the published vectors of Philox4x32-10."""
    assert philox([0], 0, 0, 0)[0].tolist() == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    f = 2 ** 64 - 1
    assert philox([0xFFFFFFFF], 0xFFFFFFFF, f, f)[0].tolist() == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    pi = philox([0x243F6A88], 0x85A308D3, 0x0370734413198A2E, 0x299F31D0A4093822)[0].tolist()
    assert pi == [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(wt._LIB_PATH):
        pytest.skip("libwtconv.so not built")
    return wt.load_library()


def _d(**kw):
    d = dict(B=2, C=16, H=4, W=4, h_dtype=1, h_layout=1, y_dtype=1, y_layout=0, norm=1, eps=1e-6, gate=0, drop=0,
             p=0.0, site=0)
    d.update(kw)
    return wt.WTConvBlockDesc(**d)


P = [ctypes.c_void_p((i + 1) << 24) for i in range(16)]   # never dereferenced: validation fails first


def _residual(lib, d, x=P[0], h=P[1], w=None, b=None, gate=None, xs=None, rng=None, out=P[2]):
    return lib.wtconv_residual_fwd(ctypes.byref(d), x, h, w, b, gate, xs, rng, out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(C=0), 1), (dict(H=0), 1), (dict(W=-3), 1), (dict(h_dtype=2), 1), (dict(y_dtype=-1), 1),
    (dict(h_layout=2), 1), (dict(y_layout=9), 1), (dict(norm=3), 1), (dict(norm=-1), 1), (dict(eps=0.0), 1),
    (dict(eps=-1e-6), 1), (dict(eps=1e-40), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(gate=3), 1),
    (dict(drop=4), 1), (dict(drop=1, p=-0.1), 1), (dict(drop=1, p=1.01), 1), (dict(drop=2, p=float("nan")), 1),
    (dict(drop=1, p=0.1, site=-1), 1), (dict(H=1 << 16, W=1 << 15), 2), (dict(B=1 << 20, C=1 << 12), 2),
    (dict(drop=1, p=0.1, B=1 << 14, C=8, H=512, W=512), 2),   # 2^32 groups
])
def test_bad_descriptors(lib, kw, status):
    d = _d(**kw)
    assert _residual(lib, d, rng=P[5]) == status
    assert lib.wtconv_residual_bwd(ctypes.byref(d), *P[:3], None, None, None, None, P[3], *[None] * 6, P[4], 1 << 30,
                                   None) == status
    assert lib.wtconv_block_workspace_size(ctypes.byref(d)) == ctypes.c_size_t(-1).value
    assert lib.wtconv_block_route(ctypes.byref(d)) == -1
    if kw.get("drop") is None and kw.get("gate") is None and kw.get("norm") is None:
        assert lib.wtconv_norm_fwd(ctypes.byref(d), P[0], None, None, P[1], None) == status
    assert lib.wtconv_norm_fwd(None, P[0], None, None, P[1], None) == 1
    assert lib.wtconv_norm_bwd(None, *P[:2], None, P[2], None, None, P[3], 1 << 20, None) == 1
    assert lib.wtconv_dropout(None, P[0], P[1], P[2], None) == 1


def test_refused_arguments(lib):
    ok = _d()
    odd = ctypes.c_void_p((1 << 24) + 1)
    for kw in (dict(x=None), dict(h=None), dict(out=None), dict(x=odd), dict(h=odd), dict(out=odd), dict(gate=P[3]),
               dict(w=ctypes.c_void_p((1 << 25) + 2)), dict(out=P[0]), dict(out=P[1]),
               dict(out=ctypes.c_void_p((1 << 24) + 1022)), dict(w=P[2]), dict(xs=P[2])):
        assert _residual(lib, ok, **kw) == 1, kw
    none = _d(norm=0)
    assert _residual(lib, none, w=P[3]) == 1 and _residual(lib, none, b=P[3]) == 1    # affine without a norm
    assert _residual(lib, _d(gate=1)) == 1                                             # the gate is missing
    assert _residual(lib, _d(drop=1, p=0.5)) == 1                                      # rng is missing
    assert _residual(lib, _d(drop=1, p=0.5), rng=ctypes.c_void_p((1 << 26) + 4)) == 1  # rng misaligned
    # the norm takes neither gate nor drop, and needs a norm
    for d in (_d(gate=1), _d(drop=2, p=0.1), none):
        assert lib.wtconv_norm_fwd(ctypes.byref(d), P[0], None, None, P[1], None) == 1
        assert lib.wtconv_norm_bwd(ctypes.byref(d), *P[:2], None, P[2], None, None, P[3], 1 << 30, None) == 1
    # dropout: a drop, an rng, no norm, no overlap
    for d, x, rng, y in ((ok, *P[:3]), (_d(norm=0), *P[:3]), (_d(norm=0, drop=1), P[0], None, P[2]),
                         (_d(norm=0, drop=1), P[0], P[1], P[0]), (_d(norm=0, drop=1), None, P[1], P[0])):
        assert lib.wtconv_dropout(ctypes.byref(d), x, rng, y, None) == 1


def test_refused_backward_arguments(lib):
    def call(d, x=None, h=P[0], dout=P[1], w=None, b=None, gate=None, xs=None, rng=None, dx=None, dh=P[2], dw=None,
             db=None, dg=None, ds=None, ws=P[3], n=1 << 23):
        return lib.wtconv_residual_bwd(ctypes.byref(d), x, h, dout, w, b, gate, xs, rng, dx, dh, dw, db, dg, ds, ws, n,
                                       None)

    ok = _d()
    need = lib.wtconv_block_workspace_size(ctypes.byref(ok))
    assert 0 < need < 1 << 22
    assert call(ok, n=need - 1) == 3 and call(ok, ws=None) == 3
    assert call(ok, ws=ctypes.c_void_p((1 << 27) + 16)) == 3
    for kw in (dict(h=None), dict(dout=None), dict(ds=P[4]), dict(dg=P[4]), dict(dh=P[0]), dict(dh=P[1]),
               dict(dx=P[2]), dict(dw=P[4], db=P[4]), dict(ws=P[1]), dict(dw=P[3])):
        assert call(ok, **kw) == 1, kw
    assert call(_d(norm=0), dw=P[4]) == 1


def test_workspace_grows_with_the_rows_only_so_far(lib):
    """The partial sums are bounded: they stay well under the activations for long inputs."""
    for cl in (0, 1):
        d = _d(B=64, C=96, H=56, W=56, h_layout=cl, y_layout=cl, gate=2)
        n = lib.wtconv_block_workspace_size(ctypes.byref(d))
        assert 0 < n < 64 * 96 * 56 * 56 * 2
    d = _d(B=1 << 20, C=1024, H=1, W=1, gate=2)
    assert lib.wtconv_block_workspace_size(ctypes.byref(d)) < 1 << 28


@pytest.mark.parametrize("kw,fused", [
    (dict(C=8, H=1, W=4), 1), (dict(C=7), 0), (dict(H=1, W=3), 0), (dict(C=2048), 1), (dict(C=2049), 0),
    (dict(C=1, y_layout=1), 1), (dict(C=7, H=1, W=1, y_layout=1), 1), (dict(C=16384, y_layout=1), 1),
    (dict(C=16385, y_layout=1), 0), (dict(h_layout=0, C=8), 1), (dict(h_layout=0, C=8, H=1, W=2), 0),
    (dict(h_dtype=0, y_dtype=0, C=2048, H=512, W=1024), 0), (dict(h_dtype=0, y_dtype=0, C=2047, H=512, W=1024), 1),
])
def test_routes(lib, kw, fused):
    """What the register kernels cover: rows up to 16,384 channels; with a planar side 8 to 2,048 channels, four
    pixels and samples under 4 GiB in fp32."""
    assert lib.wtconv_block_route(ctypes.byref(_d(**kw))) == fused


def test_empty_batch(lib):
    """B = 0: the forward calls return without launching; parameters are still checked."""
    d = _d(B=0)
    assert _residual(lib, d, x=None, h=None, out=None) == 0
    assert _residual(lib, _d(B=0, norm=0), x=None, h=None, out=None, w=P[0]) == 1
    assert lib.wtconv_norm_fwd(ctypes.byref(d), None, None, None, None, None) == 0
    assert lib.wtconv_dropout(ctypes.byref(_d(B=0, norm=0, drop=1)), None, P[0], None, None) == 0


def test_binding_refuses_host_tensors(monkeypatch):
    monkeypatch.setattr(wt, "load_library", lambda: pytest.fail("the library must not be reached"))
    x, w, rng = torch.zeros(1, 4, 2, 2), torch.zeros(4), torch.zeros(2, dtype=torch.int64)
    for call in (lambda: bb.wtconv_norm_fwd(x), lambda: bb.wtconv_norm_bwd(x, x),
                 lambda: bb.wtconv_residual_fwd(x, x, gate=w), lambda: bb.wtconv_residual_bwd(x, x),
                 lambda: bb.wtconv_dropout(x, 0.5, rng), lambda: bb.wtconv_norm_fwd("x")):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (lambda: blk.channel_norm(x), lambda: blk.block_residual(x, x),
                 lambda: blk.counter_dropout(x, 0.5, rng), lambda: blk.ChannelNorm2d(4)(x)):
        with pytest.raises(RuntimeError, match="GPU"):
            call()


def test_modules_and_their_refusals():
    n = blk.ChannelNorm2d(6, channels_last=True)
    assert torch.equal(n.weight, torch.ones(6)) and torch.equal(n.bias, torch.zeros(6))
    assert blk.ChannelNorm2d(6, kind="rms", bias=False).bias is None
    assert not list(blk.ChannelNorm2d(6, affine=False).parameters())
    r = blk.BlockResidual2d(6, norm="rms", x_scale=True, drop="sample", p=0.1)
    assert sorted(k for k, _ in r.named_parameters()) == ["bias", "gate", "weight", "x_scale"]
    assert torch.equal(r.gate, torch.full((6,), 1e-6))
    assert not list(blk.BlockResidual2d(6, layer_scale=None).parameters())
    with pytest.raises(ValueError):
        r(torch.zeros(1, 6, 2, 2), torch.zeros(1, 6, 2, 2), gate=torch.zeros(6))
    for bad in (lambda: blk.ChannelNorm2d(0), lambda: blk.ChannelNorm2d(4, kind="batch"),
                lambda: blk.ChannelNorm2d(4, eps=0), lambda: blk.BlockResidual2d(4, norm="batch"),
                lambda: blk.BlockResidual2d(4, drop="row"), lambda: blk.CounterDropout(1.5, 0),
                lambda: blk.CounterDropout(-0.1, 0), lambda: blk.CounterDropout(0.1, 0, mode="none"),
                lambda: n(torch.zeros(1, 5, 2, 2)), lambda: n(torch.zeros(6, 2, 2))):
        with pytest.raises(ValueError):
            bad()
    x = torch.zeros(1, 4, 2, 2)
    assert blk.CounterDropout(0.5, 0).eval()(x, None) is x and blk.CounterDropout(0.0, 0)(x, None) is x


def test_package_exports_the_block_operators():
    import wavelet_convolution_amd as pkg
    for name in (*pkg._BLOCK_BINDING_NAMES, *pkg._BLOCK_NAMES):
        assert name in pkg.__all__ and callable(getattr(pkg, name))


# ------------------------------------------------------------------- GPU

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
PAIRS = [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")]
ORDERS = list(itertools.product((0, 1), (0, 1)))   # channels last: of h, of the stream

# one row of one channel; single tokens; odd channels, planes smaller than a
# vector; the stage shapes' channels; long rows; wide rows, past each kernel's
# registers; planes whose last tile holds one pixel
SHAPES = [(1, 1, 1, 1), (3, 1, 5, 7), (2, 7, 1, 1), (5, 8, 1, 1), (2, 9, 2, 3), (3, 96, 7, 7), (2, 97, 5, 13),
          (2, 384, 14, 14), (1, 130, 9, 31), (2, 16, 1, 70), (70, 33, 1, 2), (1, 200, 1, 129), (2, 768, 7, 7),
          (1, 1030, 3, 5), (2, 2056, 1, 3), (1, 4100, 2, 2)]
ROWS = [(4, 520, 1, 1), (3, 1024, 1, 5), (2, 2049, 1, 2), (2, 4096, 1, 3), (1, 8200, 1, 2), (2, 16384, 1, 1),
        (1, 16385, 1, 2), (1, 20001, 1, 1)]


def _order(t, cl):
    return t.contiguous(memory_format=torch.channels_last if cl else torch.contiguous_format)


def _make(shape, h_dt, y_dt, h_cl, y_cl, seed, level=0.5):
    g = torch.Generator().manual_seed(seed)
    B, C = shape[:2]

    def act(dt, cl):
        t = torch.randn(shape, generator=g) * torch.exp(0.5 * torch.randn(1, C, 1, 1, generator=g))
        return _order((t + level * torch.randn(1, C, 1, 1, generator=g)).to(DT[dt]), cl).cuda()

    def vec(*s):
        return torch.randn(*s, generator=g).cuda()

    return dict(h=act(h_dt, h_cl), x=act(y_dt, y_cl), dy=act(y_dt, y_cl), weight=1 + 0.2 * vec(C), bias=0.3 * vec(C),
                gate_c=0.5 * vec(C), gate_s=0.5 * vec(B, C), x_scale=1 + 0.3 * vec(C),
                rng=torch.tensor([0x1234567890ABCDEF + seed, 3 + (seed << 33)], dtype=torch.int64).cuda())


def _shape_id(s):
    return "x".join(map(str, s))


def _norm_case(shape, h_dt, y_dt, h_cl, y_cl, kind, affine):
    d = _make(shape, h_dt, y_dt, h_cl, y_cl, seed=sum(shape))
    w, b = (d["weight"], d["bias"]) if affine else (None, None)
    y = bb.wtconv_norm_fwd(d["h"], w, b, kind=kind, channels_last=bool(y_cl), dtype=DT[y_dt])
    grads = bb.wtconv_norm_bwd(d["h"], d["dy"], w, b, kind=kind, want=("dx", "dweight", "dbias"))
    torch.cuda.synchronize()
    assert y.dtype == DT[y_dt] and grads[0].dtype == DT[h_dt]
    assert wt.layout_of(y) == wt.layout_of(d["dy"]) and wt.layout_of(grads[0]) == wt.layout_of(d["h"])
    ref = Ref(d["h"], kind=kind, weight=w, bias=b, dy=d["dy"])
    check("y", y, ref.out, ref.out_bound)
    for name, got in zip(("dh", "dweight", "dbias"), grads):
        check(name, got, ref.grads[name], ref.bounds[name])


@on_gpu
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("shape", SHAPES, ids=_shape_id)
def test_norm(shape, kind):
    for i, ((h_dt, y_dt), (h_cl, y_cl)) in enumerate(itertools.product(PAIRS, ORDERS)):
        print(f"[norm] {shape} {kind} {h_dt}->{y_dt} {h_cl}->{y_cl}", flush=True)
        _norm_case(shape, h_dt, y_dt, h_cl, y_cl, kind, affine=i % 3 != 2)


@on_gpu
@pytest.mark.parametrize("shape", ROWS, ids=_shape_id)
def test_norm_wide_rows(shape):
    for (h_dt, y_dt), kind in itertools.product(PAIRS, ("layer", "rms")):
        print(f"[norm rows] {shape} {kind} {h_dt}->{y_dt}", flush=True)
        _norm_case(shape, h_dt, y_dt, 1, 1, kind, affine=True)


def _residual_case(shape, h_dt, y_dt, h_cl, y_cl, kind, gate, drop, p, xs, seed=0, edit=None):
    d = _make(shape, h_dt, y_dt, h_cl, y_cl, seed=sum(shape) + seed)
    if edit:
        edit(d)
    g = {"none": None, "channel": d["gate_c"], "sample": d["gate_s"]}[gate]
    opts = dict(kind=kind, gate=g, x_scale=d["x_scale"] if xs else None)
    if kind != "none":
        opts.update(weight=d["weight"], bias=d["bias"])
    drops = dict(drop=drop, p=p, site=5)
    out = bb.wtconv_residual_fwd(d["x"], d["h"], rng=d["rng"], **opts, **drops)
    dx, dh, grads = bb.wtconv_residual_bwd(d["dy"], d["h"], x=d["x"], rng=d["rng"], **opts, **drops)
    torch.cuda.synchronize()
    seed_, off = (int(v) for v in d["rng"].cpu())
    ref = Ref(d["h"], x=d["x"], dy=d["dy"], seed=seed_, offset=off, **opts, **drops)
    assert out.dtype == d["x"].dtype and dh.dtype == d["h"].dtype
    assert wt.layout_of(out) == wt.layout_of(d["x"]) and wt.layout_of(dh) == wt.layout_of(d["h"])
    check("out", out, ref.out, ref.out_bound)
    check("dx", dx, ref.grads["dx"], ref.bounds["dx"])
    check("dh", dh, ref.grads["dh"], ref.bounds["dh"])
    for name, got in zip(("dweight", "dbias", "dgate", "dx_scale"), grads):
        if got is not None:
            check(name, got, ref.grads[name], ref.bounds[name])
    assert (dx is d["dy"]) == (not xs)
    return d, out, dx, dh, grads


MODES = list(itertools.product(("none", "layer", "rms"), ("none", "channel", "sample"),
                               (("none", 0.0), ("element", 0.3), ("sample", 0.4)), (False, True)))


@on_gpu
@pytest.mark.parametrize("shape", SHAPES, ids=_shape_id)
def test_residual(shape):
    """Every mode, each with another pair of types and orders from shape to shape."""
    for i, (kind, gate, (drop, p), xs) in enumerate(MODES):
        i += sum(shape)
        (h_dt, y_dt), (h_cl, y_cl) = PAIRS[i % 4], ORDERS[i // 4 % 4]
        print(f"[residual] {shape} {kind} {gate} {drop} {xs} {h_dt},{y_dt} {h_cl},{y_cl}", flush=True)
        _residual_case(shape, h_dt, y_dt, h_cl, y_cl, kind, gate, drop, p, xs, seed=i)


@on_gpu
@pytest.mark.parametrize("shape", ROWS, ids=_shape_id)
def test_residual_wide_rows(shape):
    for i, (kind, gate, (drop, p), xs) in enumerate(MODES[::3] + MODES[1::7]):
        h_dt, y_dt = PAIRS[i % 4]
        print(f"[residual rows] {shape} {kind} {gate} {drop} {xs} {h_dt},{y_dt}", flush=True)
        _residual_case(shape, h_dt, y_dt, 1, 1, kind, gate, drop, p, xs, seed=i)


@on_gpu
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("shape", [(5, 24, 9, 9), (3, 100, 17, 33), (64, 16, 3, 3), (2, 64, 40, 41), (9, 72, 1, 300)],
                         ids=_shape_id)
def test_residual_many_rows(shape, order):
    """Samples that end inside a workgroup's rows and samples that several workgroups share: the gate's gradient per
    sample, and the parameters' over all."""
    for gate, drop in itertools.product(("channel", "sample"), (("element", 0.5), ("sample", 0.5))):
        print(f"[many rows] {shape} {order} {gate} {drop}", flush=True)
        _residual_case(shape, "bf16", "bf16", *order, "layer", gate, *drop, True)


# grids that fill the card, where lanes hold eight bf16 pixels: four, eight and
# sixteen channel lanes, one to eight wavefronts, vectors that share elements at
# the end of channels, of pixels and of both, workgroups with several tiles of
# several samples, and several workgroups to a sample
FULL = [(350, 96, 9, 13), (350, 90, 8, 14), (1030, 30, 9, 13), (1030, 16, 3, 5), (520, 65, 7, 8), (520, 64, 7, 7),
        (520, 200, 4, 8), (520, 203, 5, 5), (130, 1000, 5, 6), (530, 1000, 3, 4), (5, 72, 90, 97)]


@on_gpu
@pytest.mark.parametrize("order", [o for o in ORDERS if o != (1, 1)])
@pytest.mark.parametrize("shape", FULL, ids=_shape_id)
def test_full_grids(shape, order):
    n = sum(shape) + 7 * order[0] + 13 * order[1]
    print(f"[full norm] {shape} {order}", flush=True)
    _norm_case(shape, "bf16", "bf16", *order, "layer" if n % 3 else "rms", affine=n % 4 > 0)
    for i in range(3):   # one of each drop
        kind, gate, (drop, p), xs = MODES[(n * 5 + 20 * i) % len(MODES)]
        print(f"[full residual] {shape} {order} {kind} {gate} {drop} {xs}", flush=True)
        _residual_case(shape, "bf16", "bf16", *order, kind, gate, drop, p, xs, seed=i)


# what the register kernels do not cover: fewer channels than a group, fewer
# pixels than a vector, more channels than a tile's; rows of a sample in one
# and in several workgroups, more rows than the workgroups' first shares
GENERIC = [(64, 7, 20, 21), (3, 5, 1, 2000), (40, 302, 1, 2), (700, 3, 2, 3), (4, 2500, 14, 14), (9, 6, 30, 31),
           (2, 3, 600, 500), (300, 1, 3, 3)]


@on_gpu
@pytest.mark.parametrize("order", [o for o in ORDERS if o != (1, 1)])
@pytest.mark.parametrize("shape", GENERIC, ids=_shape_id)
def test_generic_sizes(shape, order):
    n = sum(shape) + 7 * order[0] + 13 * order[1]
    for i in range(6):
        kind, gate, (drop, p), xs = MODES[(n * 5 + 11 * i) % len(MODES)]
        h_dt, y_dt = PAIRS[(n + i) % 4]
        print(f"[generic] {shape} {order} {kind} {gate} {drop} {xs} {h_dt} {y_dt}", flush=True)
        _residual_case(shape, h_dt, y_dt, *order, kind, gate, drop, p, xs, seed=i)
    _norm_case(shape, *PAIRS[n % 4], *order, ("layer", "rms")[n % 2], affine=True)


@on_gpu
def test_few_samples_over_many_workgroups():
    """A sample's tiles lie in many workgroups, and a workgroup's tiles in two samples."""
    for order in ((1, 0), (0, 1)):
        print(f"[shared samples] {order}", flush=True)
        _residual_case((5, 1000, 61, 57), "bf16", "bf16", *order, "layer", "sample", "element", 0.3, True)


@on_gpu
@pytest.mark.parametrize("shape", SHAPES + ROWS[-2:], ids=_shape_id)
def test_dropout(shape):
    for dt, cl, (mode, p) in itertools.product(("bf16", "f32"), (0, 1), (("element", 0.25), ("sample", 0.5))):
        print(f"[dropout] {shape} {dt} {cl} {mode}", flush=True)
        d = _make(shape, dt, dt, cl, cl, seed=sum(shape))
        y = bb.wtconv_dropout(d["h"], p, d["rng"], site=9, mode=mode)
        torch.cuda.synchronize()
        seed, off = (int(v) for v in d["rng"].cpu())
        mask, k = keep_mask(shape, mode, p, seed, off, 9)
        ref = torch.where(mask, d["h"].double().cpu() * k, torch.zeros(()).double())
        assert torch.equal((y != 0).cpu() | (d["h"].cpu() == 0), mask | (d["h"].cpu() == 0))
        check("y", y, ref, 2.0 ** -23 * ref.abs())


@on_gpu
@pytest.mark.parametrize("p,kept", [(0.0, 1.0), (2.0 ** -18, 1.0), (2.0 ** -17, None), (1 - 2.0 ** -18, 0.0), (1.0, 0.0)])
def test_dropout_borders(p, kept):
    """p rounds to 1/65536: below half a step nothing is dropped, and the values stay as they are; at one (and a
    quarter step below) everything is."""
    d = _make((2, 40, 33, 31), "f32", "f32", 1, 1, seed=1)
    for mode in ("element", "sample"):
        y = bb.wtconv_dropout(d["h"], p, d["rng"], mode=mode)
        if kept is not None:
            assert torch.equal(y, d["h"] * kept)
        else:
            seed, off = (int(v) for v in d["rng"].cpu())
            mask, _ = keep_mask(d["h"].shape, mode, p, seed, off, 0)
            assert torch.equal((y != 0).cpu(), mask & (d["h"] != 0).cpu())


@on_gpu
def test_dropout_rate_and_streams():
    """The share kept is binomial (within five deviations); another seed, offset or site is another mask."""
    x = torch.ones(4, 64, 64, 64, device="cuda")
    n = x.numel()
    masks = []
    for seed, off, site in ((1, 0, 0), (2, 0, 0), (1, 1, 0), (1, 0, 1), (1 + (1 << 32), 0, 0), (1, 1 << 32, 0)):
        rng = torch.tensor([seed, off], device="cuda")
        m = bb.wtconv_dropout(x, 0.3, rng, site=site) != 0
        T = int(0.3 * 65536 + 0.5)
        want = 1 - T / 65536
        assert abs(float(m.double().mean()) - want) < 5 * (want * (1 - want) / n) ** 0.5
        masks.append(m)
    for a, b in itertools.combinations(masks, 2):
        assert abs(float((a == b).double().mean()) - (0.49 + 0.09)) < 0.01


@on_gpu
def test_mask_is_the_same_in_every_order_and_operator():
    """The mask belongs to the element's place: the same in either memory order, type, and in the residual."""
    d = _make((3, 50, 11, 13), "f32", "bf16", 0, 0, seed=2)
    one = torch.ones_like(d["h"])
    ys = [bb.wtconv_dropout(_order(one, cl).to(dt), 0.4, d["rng"], site=3) != 0
          for cl, dt in itertools.product((0, 1), (torch.float32, torch.bfloat16))]
    out = bb.wtconv_residual_fwd(torch.zeros_like(one), one, drop="element", p=0.4, rng=d["rng"], site=3)
    for y in ys[1:] + [out != 0]:
        assert torch.equal(ys[0], y)


@on_gpu
@pytest.mark.parametrize("order", ORDERS)
def test_rows_where_nothing_is_left(order):
    """Everything dropped: the residual is x_scale x exactly, and no gradient reaches h or the parameters; h's NaN
    and infinities do not show."""
    def poison(d):
        d["h"][:, ::3] = float("nan")
        d["h"][:, 1::3] = float("inf")

    for drop in ("element", "sample"):
        d = _make((3, 24, 5, 7), "bf16", "f32", *order, seed=4)
        if drop == "sample":
            poison(d)
        opts = dict(kind="layer", weight=d["weight"], bias=d["bias"], gate=d["gate_s"], x_scale=d["x_scale"],
                    drop=drop, p=1.0, rng=d["rng"])
        out = bb.wtconv_residual_fwd(d["x"], d["h"], **opts)
        assert torch.equal(out, d["x"] * d["x_scale"].view(1, -1, 1, 1))
        dx, dh, grads = bb.wtconv_residual_bwd(d["dy"], d["h"], x=d["x"], **opts)
        for t in (dh, *grads[:3]):
            assert torch.equal(t, torch.zeros_like(t))
    y = bb.wtconv_dropout(d["h"], 1.0, d["rng"])
    assert torch.equal(y, torch.zeros_like(y))


@on_gpu
@pytest.mark.parametrize("order", ORDERS)
def test_dropped_samples_do_not_count(order):
    """A dropped sample full of NaN leaves the others' results and every parameter gradient as they are."""
    shape = (8, 40, 6, 7)
    d = _make(shape, "bf16", "bf16", *order, seed=6)
    seed, off = (int(v) for v in d["rng"].cpu())
    mask, _ = keep_mask(shape, "sample", 0.5, seed, off, 5)
    gone = ~mask[:, 0, 0, 0]
    assert 0 < int(gone.sum()) < 8

    def poison(d):
        d["h"][gone.cuda()] = float("nan")

    for kind, gate in (("layer", "sample"), ("rms", "channel"), ("none", "channel")):
        _residual_case(shape, "bf16", "bf16", *order, kind, gate, "sample", 0.5, True,
                       seed=6 - sum(shape), edit=poison)


@on_gpu
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("shape", [(3, 24, 5, 7), (2, 5, 3, 3), (4, 17, 8, 8), (1030, 16, 3, 5)], ids=_shape_id)
def test_dropped_elements_do_not_count(shape, order):
    """Without a norm a dropped element's h is not looked at: NaN and infinities there show in no result."""
    def poison(d):
        seed, off = (int(v) for v in d["rng"].cpu())
        mask, _ = keep_mask(shape, "element", 0.4, seed, off, 5)
        bad = torch.where(torch.rand(shape, generator=torch.Generator().manual_seed(1)) < 0.5, float("nan"),
                          float("inf")).to(d["h"].dtype)
        d["h"].copy_(torch.where(mask, d["h"].cpu(), bad))
        y = bb.wtconv_dropout(d["h"], 0.4, d["rng"], site=5)
        assert bool(y.isfinite().all())

    for gate, (h_dt, y_dt) in itertools.product(("channel", "sample"), PAIRS):
        _residual_case(shape, h_dt, y_dt, *order, "none", gate, "element", 0.4, True, edit=poison)


@on_gpu
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_special_rows(kind, order):
    """Rows of zeros, of one value (no variance), far from zero, of the type's lowest value, with an infinity or a
    NaN: each keeps to itself."""
    shape = (1, 72, 3, 9)
    d = _make(shape, "f32", "f32", *order, seed=8)
    h = d["h"].cpu()
    h[0, :, 0, 0] = 0
    h[0, :, 0, 1] = 2.5
    h[0, :, 0, 2] += 1000
    h[0, 5, 1, 0] = float("inf")
    h[0, 6, 1, 1] = float("nan")
    h[0, :, 2, 0] = torch.finfo(torch.float32).min
    h = _order(h, order[0]).cuda()
    y = bb.wtconv_norm_fwd(h, d["weight"], d["bias"], kind=kind, channels_last=bool(order[1]))
    dx, _, _ = bb.wtconv_norm_bwd(h, d["dy"], d["weight"], d["bias"], kind=kind)
    bad = torch.zeros(3, 9, dtype=torch.bool)
    bad[1, 0] = bad[1, 1] = bad[2, 0] = True
    ok = torch.where(bad, torch.zeros(()), h.cpu())
    ref = Ref(ok, kind=kind, weight=d["weight"], bias=d["bias"], dy=d["dy"])
    good = (~bad).expand(shape)
    zero = torch.zeros(()).double()
    check("y", torch.where(good.cuda(), y, zero.cuda()).float(), torch.where(good, ref.out, zero), ref.out_bound)
    check("dx", torch.where(good.cuda(), dx, zero.cuda()).float(), torch.where(good, ref.grads["dh"], zero),
          ref.bounds["dh"])
    assert bool(y[0, :, 1, 1].isnan().all()) and bool(y[0, 5, 1, 0].isnan())


@on_gpu
@pytest.mark.parametrize("order", ORDERS)
def test_results_repeat_bit_for_bit(order):
    d = _make((6, 90, 21, 19), "bf16", "bf16", *order, seed=9)
    opts = dict(kind="layer", weight=d["weight"], bias=d["bias"], gate=d["gate_s"], x_scale=d["x_scale"],
                drop="element", p=0.2, rng=d["rng"])

    def run():
        dx, dh, g = bb.wtconv_residual_bwd(d["dy"], d["h"], x=d["x"], **opts)
        return [bb.wtconv_residual_fwd(d["x"], d["h"], **opts), dx, dh, *g]

    first = run()
    for _ in range(3):
        for a, b in zip(first, run()):
            assert torch.equal(a, b)


@on_gpu
def test_gradients_against_differences():
    """Central differences of a weighted sum of the outputs, in the direction of random changes."""
    d = _make((2, 24, 3, 5), "f32", "f32", 1, 0, seed=10)
    fixed = dict(kind="layer", drop="element", p=0.25, rng=d["rng"], site=2)
    names = ["x", "h", "weight", "bias", "gate", "x_scale"]
    vals = dict(x=d["x"], h=d["h"], weight=d["weight"], bias=d["bias"], gate=d["gate_s"], x_scale=d["x_scale"])
    dx, dh, grads = bb.wtconv_residual_bwd(d["dy"], **{k: v for k, v in vals.items()}, **fixed)
    got = dict(zip(names, (dx, dh, *grads)))

    def loss(v):
        return float((bb.wtconv_residual_fwd(v.pop("x"), v.pop("h"), **v, **fixed).double() * d["dy"].double()).sum())

    g = torch.Generator(device="cuda").manual_seed(1)
    for n in names:
        e = torch.randn(vals[n].shape, generator=g, device="cuda").contiguous(
            memory_format=torch.channels_last if n == "h" else torch.contiguous_format)
        step = 2.0 ** -6
        diff = (loss({**vals, n: vals[n] + step * e}) - loss({**vals, n: vals[n] - step * e})) / (2 * step)
        want = float((got[n].double() * e.double()).sum())
        # the third derivative's term (step^2) and fp32 rounding of the outputs over the step
        size = float((got[n].double() * e.double()).abs().sum())
        assert abs(diff - want) <= 2e-3 * size + 1e-3, (n, diff, want)


@on_gpu
def test_given_outputs_and_workspace_and_what_is_not_wanted():
    d = _make((2, 48, 6, 5), "bf16", "f32", 1, 0, seed=11)
    ws = torch.empty(bb.wtconv_block_workspace_size(d["x"], d["h"], kind="layer", gate=d["gate_s"]) + 256,
                     dtype=torch.uint8, device="cuda")
    opts = dict(kind="layer", weight=d["weight"], bias=d["bias"], gate=d["gate_s"], x_scale=d["x_scale"])
    out = torch.full_like(d["x"], float("nan"))
    assert bb.wtconv_residual_fwd(d["x"], d["h"], out=out, **opts) is out
    dx0, dh0, g0 = bb.wtconv_residual_bwd(d["dy"], d["h"], x=d["x"], **opts)
    dx, dh = torch.full_like(d["x"], float("nan")), torch.full_like(d["h"], float("nan"))
    got = bb.wtconv_residual_bwd(d["dy"], d["h"], x=d["x"], dx=dx, dh=dh, ws=ws, **opts)
    assert got[0] is dx and got[1] is dh
    for a, b in zip((dx0, dh0, *g0), (dx, dh, *got[2])):
        assert torch.equal(a, b)
    alone = dict(zip(bb.GRADS, (dx0, dh0, *g0)))
    for n in bb.GRADS:
        dx, dh, g = bb.wtconv_residual_bwd(d["dy"], d["h"], x=d["x"], want=(n,), **opts)
        for m, t in zip(bb.GRADS, (dx, dh, *g)):
            assert (t is None) == (m != n) and (t is None or torch.equal(t, alone[n]))
    # a copy of dout where a dx is given without an x_scale
    opts["x_scale"] = None
    dx = torch.empty_like(d["x"])
    assert bb.wtconv_residual_bwd(d["dy"], d["h"], dx=dx, **opts)[0] is dx and torch.equal(dx, d["dy"])
    for a, b, c in ((None, None, ("dx",)), (d["weight"], None, ("dweight",)), (None, d["bias"], ("dbias", "dx"))):
        r = bb.wtconv_norm_bwd(d["h"], d["dy"], a, b, want=c)
        assert [t is not None for t in r] == [n in c for n in ("dx", "dweight", "dbias")]


@on_gpu
def test_binding_checks_on_the_gpu():
    d = _make((2, 8, 4, 4), "bf16", "f32", 0, 0, seed=12)
    x, h, w, rng = d["x"], d["h"], d["weight"], d["rng"]
    for bad in (lambda: bb.wtconv_norm_fwd(h[0]), lambda: bb.wtconv_norm_fwd(h.half()),
                lambda: bb.wtconv_norm_fwd(h.transpose(2, 3)), lambda: bb.wtconv_norm_fwd(h[:, :, ::2]),
                lambda: bb.wtconv_norm_fwd(h, w[:4]), lambda: bb.wtconv_norm_fwd(h, w.double()),
                lambda: bb.wtconv_norm_fwd(h, w.cpu()), lambda: bb.wtconv_norm_fwd(h, kind="none_such"),
                lambda: bb.wtconv_norm_fwd(h, y=h[:1]), lambda: bb.wtconv_norm_fwd(h, y=x, dtype=torch.bfloat16),
                lambda: bb.wtconv_norm_fwd(h, y=x, channels_last=True),
                lambda: bb.wtconv_norm_bwd(h, x[:1]), lambda: bb.wtconv_norm_bwd(h, x, dx=x),
                lambda: bb.wtconv_norm_bwd(h, x, want=("dgate",)),
                lambda: bb.wtconv_residual_fwd(x, h[:, :4]), lambda: bb.wtconv_residual_fwd(x, h, weight=w),
                lambda: bb.wtconv_residual_fwd(x, h, gate=d["gate_s"][:1]),
                lambda: bb.wtconv_residual_fwd(x, h, gate=w.view(1, 8, 1, 1)),
                lambda: bb.wtconv_residual_fwd(x, h, drop="element", p=0.1),
                lambda: bb.wtconv_residual_fwd(x, h, drop="element", p=0.1, rng=rng.int()),
                lambda: bb.wtconv_residual_fwd(x, h, drop="element", p=0.1, rng=rng[:1]),
                lambda: bb.wtconv_residual_fwd(x, h, drop="element", p=0.1, rng=rng, site=-1),
                lambda: bb.wtconv_residual_fwd(x, h, drop="rows"), lambda: bb.wtconv_residual_fwd(x, h, out=h),
                lambda: bb.wtconv_residual_bwd(x, h, x_scale=w), lambda: bb.wtconv_residual_bwd(x, h, want=("dgate",)),
                lambda: bb.wtconv_residual_bwd(x, h, want=("dweight",)),
                lambda: bb.wtconv_residual_bwd(x, h, x=h, x_scale=w), lambda: bb.wtconv_residual_bwd(x, h, dx=h),
                lambda: bb.wtconv_residual_bwd(x, h, dh=x), lambda: bb.wtconv_dropout(h, 0.5, None),
                lambda: bb.wtconv_dropout(h, 0.5, rng.float()), lambda: bb.wtconv_dropout(h, 0.5, rng, mode="none"),
                lambda: bb.wtconv_dropout(h, 0.5, rng, y=x)):
        with pytest.raises(ValueError):
            bad()
    for bad, status in ((lambda: bb.wtconv_dropout(h, 1.5, rng), 1), (lambda: bb.wtconv_dropout(h, 0.5, rng, y=h), 1),
                        (lambda: bb.wtconv_residual_fwd(x, h, out=x), 1), (lambda: bb.wtconv_norm_fwd(h, eps=0.0), 1),
                        (lambda: bb.wtconv_norm_fwd(h, eps=float("nan")), 1),
                        (lambda: bb.wtconv_norm_bwd(h, x, ws=torch.empty(16, dtype=torch.uint8, device="cuda")), 3)):
        with pytest.raises(wt.WTConvError) as e:
            bad()
        assert e.value.status == status


@on_gpu
def test_empty_batch_on_the_gpu():
    d = _make((0, 12, 3, 3), "bf16", "f32", 1, 0, seed=0)
    opts = dict(kind="rms", weight=d["weight"], bias=d["bias"], x_scale=d["x_scale"], drop="element", p=0.1,
                rng=d["rng"])
    for gate in (d["gate_c"], d["gate_s"]):
        assert bb.wtconv_residual_fwd(d["x"], d["h"], gate=gate, **opts).shape == d["x"].shape
        dx, dh, grads = bb.wtconv_residual_bwd(d["dy"], d["h"], x=d["x"], gate=gate, **opts)
        assert dx.shape == d["x"].shape and dh.shape == d["h"].shape
        for t, like in zip(grads, (d["weight"], d["bias"], gate, d["x_scale"])):
            assert torch.equal(t, torch.zeros_like(like))
    assert bb.wtconv_dropout(d["h"], 0.1, d["rng"]).shape == d["h"].shape


@on_gpu
def test_misaligned_views():
    """Samples of an odd size start at addresses aligned to the element only."""
    big = _make((3, 7, 3, 5), "bf16", "bf16", 0, 0, seed=13)
    h, x, dy = (big[n][1:] for n in ("h", "x", "dy"))
    assert h.data_ptr() % 4 == 2 and h.is_contiguous()
    opts = dict(kind="layer", weight=big["weight"], bias=big["bias"], gate=big["gate_c"])
    clones = [t.clone() for t in (x, h, dy)]
    assert torch.equal(bb.wtconv_residual_fwd(x, h, **opts), bb.wtconv_residual_fwd(*clones[:2], **opts))
    a, b = bb.wtconv_residual_bwd(dy, h, **opts), bb.wtconv_residual_bwd(clones[2], clones[1], **opts)
    for s, t in zip((a[1], *a[2][:3]), (b[1], *b[2][:3])):
        assert torch.equal(s, t)
    assert torch.equal(bb.wtconv_dropout(h, 0.5, big["rng"]), bb.wtconv_dropout(clones[1], 0.5, big["rng"]))


@on_gpu
def test_another_stream():
    """Calls on a stream that is not current, with outputs and workspace allocated there, and inputs dropped while it
    still runs."""
    d = _make((16, 96, 28, 28), "bf16", "bf16", 1, 0, seed=14)
    opts = dict(kind="layer", weight=d["weight"], bias=d["bias"], gate=d["gate_c"], x_scale=d["x_scale"])
    want = [bb.wtconv_residual_fwd(d["x"], d["h"], **opts), bb.wtconv_residual_bwd(d["dy"], d["h"], x=d["x"], **opts)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x, h, dy = d["x"].clone(), d["h"].clone(), d["dy"].clone()
    s.wait_stream(torch.cuda.current_stream())
    out = bb.wtconv_residual_fwd(x, h, stream=s, **opts)
    dx, dh, grads = bb.wtconv_residual_bwd(dy, h, x=x, stream=s, **opts)
    del x, h, dy
    junk = [torch.full_like(d["x"], 7.0) for _ in range(6)]
    s.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(dx, want[1][0]) and torch.equal(dh, want[1][1])
    for a, b in zip(grads, want[1][2]):
        assert torch.equal(a, b)
    del junk


@on_gpu
def test_two_streams_at_once():
    """Calls that run side by side on two streams share nothing."""
    ds = [_make((32, 96, 28, 28), "bf16", "bf16", 1, 0, seed=k) for k in (20, 21)]

    def run(d, s):
        opts = dict(kind="layer", weight=d["weight"], bias=d["bias"], gate=d["gate_s"], x_scale=d["x_scale"],
                    drop="element", p=0.2, rng=d["rng"], stream=s)
        dx, dh, g = bb.wtconv_residual_bwd(d["dy"], d["h"], x=d["x"], **opts)
        return [bb.wtconv_residual_fwd(d["x"], d["h"], **opts), dx, dh, *g]

    want = [run(d, None) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    got = [[run(d, s) for d, s in zip(ds, streams)] for _ in range(8)]
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            for t, u in zip(a, b):
                assert torch.equal(t, u)


@on_gpu
def test_captured_and_replayed():
    """Forward, backward and dropout captured in one graph: every replay equals the eager calls for the values that
    its inputs hold then, the generator's state among them; a second graph of the same calls shares nothing."""
    d = _make((4, 96, 14, 14), "bf16", "bf16", 1, 0, seed=15)
    opts = dict(kind="rms", weight=d["weight"], bias=d["bias"], gate=d["gate_s"], x_scale=d["x_scale"],
                drop="element", p=0.3, rng=d["rng"], site=1)

    def step():
        u = bb.wtconv_norm_fwd(d["x"], d["weight"], d["bias"], channels_last=True)
        h = bb.wtconv_dropout(u, 0.2, d["rng"], site=2)
        out = bb.wtconv_residual_fwd(d["x"], h, **opts)
        dx, dh, g = bb.wtconv_residual_bwd(d["dy"], h, x=d["x"], **opts)
        n = bb.wtconv_norm_bwd(d["x"], bb.wtconv_dropout(dh, 0.2, d["rng"], site=2), d["weight"], d["bias"])
        return [out, dx, dh, *g, *n]

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
        graphs.append((g, got))
    masks = []
    for k in range(3):
        d["rng"][1] += 1
        d["x"].copy_(torch.randn_like(d["x"]))
        want = step()
        torch.cuda.synchronize()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, got in graphs:
            for a, b in zip(got, want):
                assert torch.equal(a, b)
        masks.append(want[2] != 0)
    assert not torch.equal(masks[0], masks[1])


@on_gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_block_as_used(dt):
    """Norm, MLP dropout, and residual around a WTConv mixer, through the modules: outputs and gradients against the
    same block in 64 bits (the mixer and the matrix products are the run's own outputs there)."""
    torch.manual_seed(0)
    B, C, H = 3, 24, 14
    from wavelet_convolution_amd import WTConv2d
    mixer = WTConv2d(C, 1, device="cuda")
    norm = blk.ChannelNorm2d(C, channels_last=True, device="cuda")
    drop = blk.CounterDropout(0.2, site=1)
    end = blk.BlockResidual2d(C, norm="rms", layer_scale=0.3, x_scale=True, drop="sample", p=0.4, site=2,
                              device="cuda")
    rng = blk.dropout_rng(77)
    x = torch.randn(B, C, H, H, device="cuda").to(DT[dt]).requires_grad_()
    a = mixer(x)
    u = norm(a)
    rows = u.permute(0, 2, 3, 1)
    assert rows.is_contiguous()
    h = drop(torch.nn.functional.gelu(rows).permute(0, 3, 1, 2), rng)
    out = end(x, h, rng)
    for t in (a, u, h):
        t.retain_grad()
    dy = torch.randn_like(out)
    out.backward(dy)
    torch.cuda.synchronize()
    seed = int(rng[0])
    r = Ref(h, x=x, kind="rms", weight=end.weight, bias=end.bias, gate=end.gate, x_scale=end.x_scale, drop="sample",
            p=0.4, seed=seed, site=2, dy=dy)
    check("out", out, r.out, r.out_bound)
    check("dh", h.grad, r.grads["dh"], r.bounds["dh"])
    for n, q in (("dweight", end.weight), ("dbias", end.bias), ("dgate", end.gate), ("dx_scale", end.x_scale)):
        check(n, q.grad, r.grads[n], r.bounds[n])
    n = Ref(a, kind="layer", weight=norm.weight, bias=norm.bias, dy=u.grad)
    check("u", u, n.out, n.out_bound)
    check("da", a.grad, n.grads["dh"], n.bounds["dh"])
    check("norm dweight", norm.weight.grad, n.grads["dweight"], n.bounds["dweight"])
    assert x.grad is not None and bool(x.grad.isfinite().all())
    # autograd refuses a state that changed between the passes
    y = drop(x, rng)
    rng[1] += 1
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.sum().backward()
    # eval mode drops nothing
    for m in (drop, end):
        m.eval()
    assert drop(x, None) is x
    full = Ref(h, x=x, kind="rms", weight=end.weight, bias=end.bias, gate=end.gate, x_scale=end.x_scale)
    check("eval", end(x, h), full.out, full.out_bound)


@on_gpu
def test_training_step_captured():
    """Norm, dropout, residual and their backward through autograd in one graph, with the generator's step inside:
    every replay equals the eager step for the same state, and the masks move on."""
    B, C, H = 4, 32, 14
    torch.manual_seed(1)
    norm = blk.ChannelNorm2d(C, channels_last=True, device="cuda")
    drop = blk.CounterDropout(0.25, site=1)
    end = blk.BlockResidual2d(C, norm="rms", layer_scale=0.5, x_scale=True, drop="sample", p=0.3, site=2,
                              device="cuda")
    rng = blk.dropout_rng(5)
    x = torch.randn(B, C, H, H, device="cuda").requires_grad_()
    dy = torch.randn(B, C, H, H, device="cuda")
    leaves = [x, *norm.parameters(), *end.parameters()]

    def step():
        out = end(x, drop(norm(x), rng), rng)
        grads = torch.autograd.grad(out, leaves, dy)
        rng[1] += 1
        return [out.detach(), *grads]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    outs = []
    for k in range(3):
        rng[1] = 10 + k
        g.replay()
        torch.cuda.synchronize()
        assert int(rng[1]) == 11 + k
        replayed = [t.clone() for t in got]
        rng[1] = 10 + k
        for a, b in zip(replayed, step()):
            assert torch.equal(a, b)
        outs.append(replayed[0])
    assert not torch.equal(outs[0], outs[1])


@on_gpu
def test_second_derivatives_are_refused():
    x = torch.randn(2, 16, 4, 4, device="cuda", requires_grad=True)
    rng = blk.dropout_rng(1)
    for fn in (lambda: blk.channel_norm(x), lambda: blk.block_residual(x, x, kind="rms"),
               lambda: blk.counter_dropout(x, 0.5, rng)):
        g, = torch.autograd.grad(fn().square().sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            g.sum().backward()


@on_gpu
def test_functions_keep_inputs_only_and_take_any_view():
    """Autograd keeps the inputs alone (no mask, no statistics, no output); strided and expanded views are copied."""
    x = torch.randn(4, 32, 14, 14, device="cuda", requires_grad=True)
    h = torch.randn(4, 14, 14, 32, device="cuda").permute(0, 3, 1, 2).requires_grad_()
    rng = blk.dropout_rng(1)
    end = blk.BlockResidual2d(32, norm="layer", drop="element", p=0.5, device="cuda")
    saved = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: saved.append(t) or t, lambda t: t):
        out = end(x, h, rng)
        out = blk.counter_dropout(blk.channel_norm(out), 0.5, rng, site=4)
    known = {t.data_ptr() for t in (h, rng, *end.parameters())}
    extra = [t for t in saved if t.data_ptr() not in known]
    assert len(extra) == 1   # the residual's output, the norm's own input
    out.sum().backward()     # an expanded gradient
    wide = torch.randn(4, 32, 14, 28, device="cuda")[..., ::2]
    assert torch.equal(blk.channel_norm(wide), blk.channel_norm(wide.contiguous()))
    row = torch.randn(1, 32, 1, 1, device="cuda").expand(4, 32, 14, 14)
    assert torch.equal(blk.block_residual(x, row), blk.block_residual(x, row.contiguous()))
    assert torch.equal(blk.counter_dropout(wide, 0.5, rng), blk.counter_dropout(wide.contiguous(), 0.5, rng))


@on_gpu
def test_long_offsets():
    """More than 2^31 elements, in rows and in planes: the last rows are right (dropout's, too)."""
    C, n = 8, (1 << 28) + 3
    rng = torch.tensor([5, 6], device="cuda")
    x = torch.zeros(1, n, C, dtype=torch.bfloat16, device="cuda")
    x[:, -5:] = torch.randn(1, 5, C, device="cuda").to(torch.bfloat16)
    rows = x.view(1, 1, n, C).permute(0, 3, 1, 2)
    y = bb.wtconv_norm_fwd(rows, kind="rms")
    ref = Ref(rows[..., -5:], kind="rms")
    check("y", y[..., -5:].contiguous(), ref.out, ref.out_bound)
    del y
    x.fill_(1)
    y = bb.wtconv_dropout(rows, 0.5, rng, site=1)
    w = philox(np.arange(n - 5, n), 1, 6, 5)
    bits = np.stack((w & 0xFFFF, w >> 16), -1).reshape(5, 8) >= 32768
    assert torch.equal((y[0, :, 0, -5:].T != 0).cpu(), torch.from_numpy(bits))
    del y, rows, x
    planes = torch.zeros(n // 4096, 8, 64, 64, dtype=torch.bfloat16, device="cuda")
    planes[-1, :, -1, -5:] = torch.randn(8, 5, device="cuda").to(torch.bfloat16)
    y = bb.wtconv_norm_fwd(planes, kind="rms", channels_last=True)
    last = planes[-1:, :, -1:, -5:].contiguous()
    ref = Ref(last, kind="rms")
    check("planes", y[-1:, :, -1:, -5:].contiguous(), ref.out, ref.out_bound)


@on_gpu
@pytest.mark.parametrize("order", [(1, 1), (0, 1), (1, 0)])
def test_long_offsets_backward(order):
    """More than 2^31 elements, all zeros but the last pixels: those pixels' gradients, and the parameters' from them
    alone."""
    C, last = 8, 5
    B, H, W = ((1 << 28) + 4096) // 4096, 64, 64
    g = torch.Generator().manual_seed(3)
    tail = {n: torch.randn(1, C, 1, last, generator=g) for n in ("h", "dy")}

    def full(cl, t):
        x = torch.zeros((B, H, W, C) if cl else (B, C, H, W), dtype=torch.bfloat16, device="cuda")
        x = x.permute(0, 3, 1, 2) if cl else x
        x[-1:, :, -1:, -last:] = t.to(torch.bfloat16).cuda()
        return x

    h, dy = full(order[0], tail["h"]), full(order[1], tail["dy"])
    w = (1 + 0.2 * torch.randn(C, generator=g)).cuda()
    gate, xs = torch.randn(C, generator=g).cuda(), torch.randn(C, generator=g).cuda()
    opts = dict(kind="rms", weight=w, gate=gate, x_scale=xs)
    dx, dh, grads = bb.wtconv_residual_bwd(dy, h, x=dy, **opts)
    ends = [t[-1:, :, -1:, -last:].contiguous() for t in (h, dy)]
    ref = Ref(ends[0], x=ends[1], dy=ends[1], **opts)
    for name, t in (("dx", dx), ("dh", dh)):
        check(name, t[-1:, :, -1:, -last:].contiguous(), ref.grads[name], ref.bounds[name])
    for name, t in zip(("dweight", "dbias", "dgate", "dx_scale"), grads):
        if t is not None:
            check(name, t, ref.grads[name], ref.bounds[name])


@on_gpu
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("shape", [(3, 24, 5, 7), (1030, 16, 3, 5), (2, 5, 3, 3), (4, 1030, 1, 6), (6, 40, 1, 1)],
                         ids=_shape_id)
def test_an_infinite_gradient_stays_infinite(shape, order):
    """Without a bias the gate's gradient sum dout D(v) is infinite, with the sign of that one product, in the
    channel where one dout is infinite, and the other channels' are as they were."""
    d = _make(shape, "bf16", "f32", *order, seed=16)
    b, c, i, j = shape[0] - 1, shape[1] // 2, shape[2] - 1, 0
    inf = d["dy"].clone()
    inf[b, c, i, j] = float("inf")
    for kind, gate in itertools.product(("none", "layer", "rms"), ("gate_c", "gate_s")):
        opts = dict(kind=kind, gate=d[gate], weight=None if kind == "none" else d["weight"], want=("dh", "dgate"))
        plain, got = (bb.wtconv_residual_bwd(dy, d["h"], **opts)[2][2].cpu() for dy in (d["dy"], inf))
        t = bb.wtconv_residual_fwd(torch.zeros_like(d["x"]), d["h"], kind=kind, weight=opts["weight"])[b, c, i, j]
        at = (c,) if gate == "gate_c" else (b, c)
        assert float(t) != 0 and float(got[at]) == float("inf") * float(t), (kind, gate, float(got[at]), float(t))
        got[at] = plain[at]
        assert torch.equal(got, plain)
