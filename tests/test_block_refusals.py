"""What the block operators and the layer refuse before anything is launched (CPU)."""
import ctypes
import os

import pytest
import torch

from wavelet_convolution_amd import binding as wt
from wavelet_convolution_amd import block_binding as bb

class NoCalls:
    """A library whose entry points must not be called."""
    def __getattr__(self, name):
        return lambda *a: pytest.fail(f"{name} must not be called")


# dimensions that 32 bits cut to 16, 1, 0 and a negative number
LONG = [(1, 1, 1, (1 << 32) + 16), ((1 << 32) + 1, 8, 1, 1), (1, 1 << 32, 1, 1), (1, 1, (1 << 31) + 5, 1)]


@pytest.mark.parametrize("shape", LONG)
def test_sizes_past_32_bits_are_refused(shape, monkeypatch):
    """No descriptor is built for a size that its fields do not hold: the binding raises before the library is
    called, for queries and calls alike (tensors without storage stand for those of many GB)."""
    monkeypatch.setattr(wt, "load_library", NoCalls)
    x = torch.empty(shape, dtype=torch.bfloat16, device="meta")
    rows = torch.empty(shape, dtype=torch.bfloat16, device="meta", memory_format=torch.channels_last)
    monkeypatch.setattr(bb, "_on_gpu", lambda *a, **k: None)
    monkeypatch.setattr(bb, "_elsewhere", lambda *a: False)
    rng = torch.zeros(2, dtype=torch.int64)
    for call in (lambda: bb._desc(x, (1, 0), (1, 0)), lambda: bb.wtconv_block_workspace_size(x, rows),
                 lambda: bb.wtconv_block_route(rows, x), lambda: bb.wtconv_norm_fwd(x),
                 lambda: bb.wtconv_norm_bwd(x, rows), lambda: bb.wtconv_residual_fwd(x, rows),
                 lambda: bb.wtconv_residual_bwd(x, rows), lambda: bb.wtconv_dropout(x, 0.5, rng),
                 lambda: wt.wtconv_workspace_size(x, 0, 5, 3, wt.OP_FWD), lambda: wt.wtconv_route(x, 0, 5, 3, wt.OP_FWD)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


@pytest.mark.parametrize("levels,k_base,k_level", [(1 << 32, 5, 5), (1, (1 << 32) + 5, 5), (1, 5, (1 << 32) + 5)])
def test_levels_and_kernels_past_32_bits_are_refused(levels, k_base, k_level, monkeypatch):
    monkeypatch.setattr(wt, "load_library", NoCalls)
    x = torch.empty((1, 8, 32, 32), device="meta")
    for fn in (wt.wtconv_workspace_size, wt.wtconv_route):
        with pytest.raises(ValueError, match="2\\^31"):
            fn(x, levels, k_base, k_level, wt.OP_FWD)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(wt._LIB_PATH):
        pytest.skip("libwtconv.so not built")
    return wt.load_library()


def _d(**kw):
    d = dict(B=1, C=16, H=1, W=1, h_dtype=1, h_layout=1, y_dtype=1, y_layout=1, norm=2, eps=1e-6, gate=0, drop=0,
             p=0.0, site=0)
    d.update(kw)
    return ctypes.byref(wt.WTConvBlockDesc(**d))


P = [ctypes.c_void_p((i + 1) << 40) for i in range(8)]   # never dereferenced: validation fails first


@pytest.mark.parametrize("h_layout,drop", [(1, 0), (0, 0), (1, 1), (1, 2)])
@pytest.mark.parametrize("C", [(1 << 30) + 1, (1 << 31) - 257, (1 << 31) - 256, (1 << 31) - 8, (1 << 31) - 1])
def test_channels_past_2_30_are_refused(lib, C, h_layout, drop):
    """The kernels step over channels in 32-bit numbers, by as much as a workgroup at once."""
    d = _d(C=C, h_layout=h_layout, drop=drop, p=0.5)
    assert lib.wtconv_block_workspace_size(d) == ctypes.c_size_t(-1).value
    assert lib.wtconv_block_route(d) == -1
    assert lib.wtconv_residual_fwd(d, P[0], P[1], None, None, None, None, P[2], P[3], None) == 2
    assert lib.wtconv_residual_bwd(d, None, P[0], P[1], None, None, None, None, P[2], None, P[3], None, None, None,
                                   None, P[4], 1 << 39, None) == 2
    if drop:
        assert lib.wtconv_dropout(_d(C=C, norm=0, h_layout=h_layout, drop=drop, p=0.5), P[0], P[2], P[3], None) == 2
    else:
        assert lib.wtconv_norm_fwd(d, P[0], None, None, P[1], None) == 2
        assert lib.wtconv_norm_bwd(d, P[0], P[1], None, P[2], None, None, P[4], 1 << 39, None) == 2


def test_channels_up_to_2_30_are_taken(lib):
    for kw in (dict(), dict(h_layout=0, H=2), dict(drop=1, p=0.5), dict(B=1, gate=2)):
        d = _d(C=1 << 30, **kw)
        assert lib.wtconv_block_route(d) == 0
        # partial sums of every wanted gradient, a slot of C numbers each at least
        assert 1 << 32 <= lib.wtconv_block_workspace_size(d) < 1 << 40


@pytest.mark.parametrize("kw,status", [(dict(kind="layer", eps=0.0), 1), (dict(kind="rms", eps=float("nan")), 1),
                                       (dict(drop="element", p=1.5), 1), (dict(drop="sample", p=-0.5), 1)])
def test_backward_calls_name_the_argument_that_is_wrong(lib, kw, status, monkeypatch):
    """A bad eps or p is an invalid argument in a backward call too (which asks for its workspace first), as it is
    forwards; the check is the library's own, on host memory that no kernel sees."""
    monkeypatch.setattr(bb, "_on_gpu", lambda *a, **k: None)
    monkeypatch.setattr(bb, "_elsewhere", lambda *a: False)
    monkeypatch.setattr(bb, "_stream", lambda act: 0)
    x, h, rng = torch.zeros(2, 16, 4, 4), torch.zeros(2, 16, 4, 4), torch.zeros(2, dtype=torch.int64)
    calls = [lambda: bb.wtconv_residual_fwd(x, h, rng=rng, **kw), lambda: bb.wtconv_residual_bwd(x, h, rng=rng, **kw)]
    if "drop" not in kw:
        calls += [lambda: bb.wtconv_norm_fwd(x, **kw), lambda: bb.wtconv_norm_bwd(x, h, **kw)]
    for call in calls:
        with pytest.raises(wt.WTConvError) as e:
            call()
        assert e.value.status == status


class _Copies(torch.utils._python_dispatch.TorchDispatchMode):
    """Counts the tensors made of as many elements as a gradient has."""
    def __init__(self, n):
        super().__init__()
        self.n, self.made = n, []

    def __torch_dispatch__(self, fn, types, args=(), kwargs=None):
        out = fn(*args, **(kwargs or {}))
        if fn._schema.name in ("aten::clone", "aten::empty", "aten::empty_like", "aten::new_empty") \
                and out.numel() == self.n:
            self.made.append(fn._schema.name)
        return out


@pytest.mark.parametrize("channels_last", [False, True])
def test_a_strided_gradient_is_copied_once(channels_last, monkeypatch):
    """The residual's backward pass copies an expanded or strided dout into the stream's order, and copies nothing
    more; one in either order is taken as it is (the call to the library is replaced)."""
    from wavelet_convolution_amd import block as blk
    got = []
    monkeypatch.setattr(bb, "wtconv_residual_bwd",
                        lambda dout, h, **kw: got.append(dout) or (dout, h, (None,) * 4))
    order = torch.channels_last if channels_last else torch.contiguous_format
    h = torch.zeros(2, 8, 4, 6)

    class Ctx:
        saved_tensors = (None, h, None, None, None, None, None)
        needs_input_grad = (True, True) + (False,) * 10
        opts = {}

    Ctx.order = order
    wide = torch.randn(2, 8, 4, 12)
    for dout, copies in ((torch.ones(()).expand(2, 8, 4, 6), 1), (wide[..., ::2], 1), (h.clone(), 0),
                         (torch.randn(2, 8, 4, 6).contiguous(memory_format=torch.channels_last), 0)):
        got.clear()
        with _Copies(h.numel()) as c:
            blk.BlockResidualFunction.backward(Ctx, dout)
        assert torch.equal(got[0], dout) and (got[0] is dout) == (copies == 0)
        assert len(c.made) == copies, c.made
        if copies:
            assert got[0].is_contiguous(memory_format=order)


def test_a_workspace_that_is_no_block_of_memory_is_refused():
    """An expanded or strided tensor counts more bytes than it owns, or leaves gaps."""
    few = torch.zeros(1, dtype=torch.uint8)
    for ws in (few.expand(1 << 20), torch.zeros(64, 64).t()[:, :3]):
        with pytest.raises(ValueError, match="ws must be contiguous"):
            wt._ws_bytes(ws)
        with pytest.raises(ValueError, match="ws must be contiguous"):
            bb._workspace(None, few, ws)
    assert 64 * 64 * 4 - 256 < wt._ws_bytes(torch.zeros(64, 64)) <= 64 * 64 * 4
