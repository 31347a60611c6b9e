"""MI355X-native WTConv: fused HIP kernels for gfx950 behind a C-ABI.

The compute path is ``libwtconv.so`` (HIP, built from ``csrc/``); the Python
functions here only marshal arguments to it. Importing the package does not
load the library; the first call of a binding function does, and raises if
the library is missing.
"""
from .configs import CONFIGS, WorkloadConfig, get_config  # noqa: F401

_BINDING_NAMES = (
    "wtconv_fwd", "wtconv_bwd_data", "wtconv_bwd_weight",
    "wtconv_naive_fwd", "wtconv_naive_bwd_data", "wtconv_naive_bwd_weight",
    "wtconv_workspace_size", "wtconv_status_string", "load_library", "WTConvError",
    "wtconv_bwd", "wtconv_peak_fma", "wtconv_peak_copy", "layout_of", "wtconv_route",
)

_MODULE_NAMES = ("WTConv2d", "WTConvFunction", "wtconv")

# the block operators around the layer: channel norm, block residual, counter dropout
_BLOCK_BINDING_NAMES = (
    "wtconv_norm_fwd", "wtconv_norm_bwd", "wtconv_residual_fwd", "wtconv_residual_bwd", "wtconv_dropout",
    "wtconv_block_workspace_size", "wtconv_block_route",
)

_BLOCK_NAMES = ("ChannelNorm2d", "BlockResidual2d", "CounterDropout", "channel_norm", "block_residual",
                "counter_dropout", "dropout_rng")

__all__ = ["CONFIGS", "WorkloadConfig", "get_config", *_BINDING_NAMES, *_MODULE_NAMES, *_BLOCK_BINDING_NAMES,
           *_BLOCK_NAMES]


def __getattr__(name):
    # the binding is imported on first use so that CPU-only code (configs,
    # inputs, the I/O model) never needs the HIP runtime
    if name in _BINDING_NAMES:
        from . import binding
        return getattr(binding, name)
    if name in _MODULE_NAMES:
        from . import module
        return getattr(module, name)
    if name in _BLOCK_BINDING_NAMES:
        from . import block_binding
        return getattr(block_binding, name)
    if name in _BLOCK_NAMES:
        from . import block
        return getattr(block, name)
    raise AttributeError(name)
