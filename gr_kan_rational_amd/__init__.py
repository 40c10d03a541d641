"""MI355X-native GR-KAN (Group-Rational KAN) safe Pade activation.

The compute path is the HIP library ``libgrkan.so`` (hand-written gfx950
kernels behind a C ABI declared in ``include/grkan.h``, for the operators
around the activation in a transformer block ``include/grkan_block.h`` and for
those of a deep stack's training step ``include/grkan_train.h``); the names
below are its thin Python binding.  Importing this package loads nothing: the library
is loaded on first use and a missing or unloadable library raises.
"""
__all__ = [
    "grkan_forward",
    "grkan_backward",
    "grkan_backward_workspace_size",
    "grkan_status_string",
    "GRKANFunction",
    "GRKANError",
    "grkan_query_launch",
    "grkan_pau_forward",
    "grkan_pau_backward",
    "grkan_pau_backward_workspace_size",
    "grkan_pau_query_launch",
    "grkan_pau_supported",
    "load_library",
]
_BLOCK = [
    "grkan_group_norm_forward",
    "grkan_group_norm_backward",
    "GRKANGroupNorm",
    "grkan_linear_act_forward",
    "grkan_linear_act_backward",
    "GRKANLinearAct",
]
_TRAIN = [
    "grkan_fp8_quantize",
    "grkan_fp8_matmul",
    "GRKANFp8Linear",
    "grkan_residual_norm_forward",
    "grkan_residual_norm_backward",
    "GRKANResidualNorm",
    "grkan_adamw_step",
    "grkan_adamw_state",
    "GRKANAdamW",
]
__all__ += _BLOCK + _TRAIN


def __getattr__(name):
    if name in _BLOCK or name in _TRAIN:
        from . import block, train

        globals()[name] = getattr(block if name in _BLOCK else train, name)  # the next access finds it without this function
        return globals()[name]
    if name in __all__:
        from . import binding

        return getattr(binding, name)
    raise AttributeError(name)
