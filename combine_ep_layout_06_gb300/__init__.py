"""GB300-native (sm_103a) MoE expert-parallel token layout, dispatch and
combine over W logical ranks held in one GPU's HBM.

The compute path is the CUDA library libep_gb300.so (C ABI in
include/ep_api.h); ``EpDispatchCombineOp`` is a thin ctypes binding over it.
The calls around it, top-k routing (``route``), the balance loss
(``balance_loss``), the experts' matrix products (``expert_product``) and the norm
(``rms_norm``), each with its gradient, activations kept in 8 bits
(``checkpoint``) and the experts of a few tokens (``moe_few_tokens``), go through
a compiled binding.
Submodules are imported lazily so that ``combine_ep_layout_06_gb300.inputs``
(the seeded input generator) can be used without loading the library.
"""
__all__ = ["EpDispatchCombineConfig", "EpDispatchCombineOp", "EpError",
           "balance_loss", "balance_loss_backward", "checkpoint",
           "checkpoint_restore", "expert_product", "expert_product_backward",
           "moe_error", "moe_few_tokens", "rms_norm", "rms_norm_backward",
           "route", "route_backward", "workspace_size"]

_MOE = ("balance_loss", "balance_loss_backward", "checkpoint",
        "checkpoint_restore", "expert_product", "expert_product_backward",
        "moe_error", "moe_few_tokens", "rms_norm", "rms_norm_backward",
        "route", "route_backward")


def __getattr__(name):
    if name in ("EpDispatchCombineConfig", "EpDispatchCombineOp",
                "workspace_size"):
        from . import op
        return getattr(op, name)
    if name in _MOE:
        from . import moe
        globals().update({n: getattr(moe, n) for n in _MOE})
        return globals()[name]
    if name == "EpError":
        from ._lib import EpError
        return EpError
    raise AttributeError(name)
