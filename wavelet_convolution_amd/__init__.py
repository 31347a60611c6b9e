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

# rows to their experts and back, and the optimizer's step over many tensors
_EXPERT_BINDING_NAMES = ("wtconv_expert_sort", "wtconv_expert_rows_fwd", "wtconv_expert_rows_bwd",
                         "wtconv_expert_sum_fwd", "wtconv_expert_sum_bwd")
_EXPERT_NAMES = ("ExpertRoute", "expert_sort", "expert_rows", "expert_sum")
_OPTIM_BINDING_NAMES = ("wtconv_adamw_step", "wtconv_adamw_check", "wtconv_adamw_state_count", "wtconv_grad_norm")
_OPTIM_NAMES = ("AdamW",)

__all__ = ["CONFIGS", "WorkloadConfig", "get_config", *_BINDING_NAMES, *_MODULE_NAMES, *_BLOCK_BINDING_NAMES,
           *_BLOCK_NAMES, *_EXPERT_BINDING_NAMES, *_EXPERT_NAMES, *_OPTIM_BINDING_NAMES, *_OPTIM_NAMES]


# the module of each name: imported on first use, so that CPU-only code
# (configs, inputs, the I/O model) never needs the HIP runtime
_HOMES = {name: home for home, names in (
    ("binding", _BINDING_NAMES), ("module", _MODULE_NAMES), ("block_binding", _BLOCK_BINDING_NAMES),
    ("block", _BLOCK_NAMES), ("expert_binding", _EXPERT_BINDING_NAMES), ("experts", _EXPERT_NAMES),
    ("optim_binding", _OPTIM_BINDING_NAMES), ("optim", _OPTIM_NAMES)) for name in names}


def __getattr__(name):
    home = _HOMES.get(name)
    if home is None:
        raise AttributeError(name)
    import importlib
    # kept: the next use does not come here
    value = globals()[name] = getattr(importlib.import_module(f".{home}", __name__), name)
    return value
