"""What the block operators and the layer refuse before anything is launched (CPU)."""
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
