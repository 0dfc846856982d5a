"""MI355X-native EMA-Gram quarter-power preconditioner step, and the operators
of the linear layers and banks of experts whose weights it updates.

The compute path is the C-ABI library ``libmatrix_roots.so`` (hand-written
HIP kernels for gfx950) declared in ``include/matrix_roots.h``; this package
is a thin ctypes binding over it.  The library is loaded on first use, and a
missing library raises instead of falling back to anything else.
"""

from __future__ import annotations

__all__ = [
    "gram_ema_update",
    "inv_quarter_root_batched",
    "precondition_apply",
    "library",
    "rms_norm_forward",
    "rms_norm_backward",
    "layer_norm_forward",
    "layer_norm_backward",
    "quantize_blocks",
    "block_scaled_matmul",
    "grouped_matmul",
    "grouped_weight_grad",
    "route_tokens",
    "route_tokens_backward",
    "order_by_expert",
    "dispatch_rows",
    "dispatch_rows_backward",
    "combine_rows",
    "combine_rows_backward",
    "Routed",
    "ExpertOrder",
    "clip_gradients_batched",
]

_LINEAR = ("rms_norm_forward", "rms_norm_backward", "layer_norm_forward", "layer_norm_backward", "quantize_blocks",
           "block_scaled_matmul", "grouped_matmul", "grouped_weight_grad")
_EXPERTS = ("route_tokens", "route_tokens_backward", "order_by_expert", "dispatch_rows", "dispatch_rows_backward",
            "combine_rows", "combine_rows_backward", "Routed", "ExpertOrder")


def __getattr__(name):
    if name in _LINEAR:
        from . import linear

        return globals().setdefault(name, getattr(linear, name))
    if name in _EXPERTS:
        from . import experts

        return globals().setdefault(name, getattr(experts, name))
    if name in __all__:
        from . import binding

        return getattr(binding, name)
    raise AttributeError(name)
