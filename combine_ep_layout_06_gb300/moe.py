"""What stands before and between dispatch and combine in a MoE layer:
``route`` (router logits -> dispatch's weights and indices), ``balance_loss``
(the loss that evens out the experts' loads, with per-expert counts) and
``expert_product`` (one matrix product per expert over the rows that
``moe_group`` leaves, with bias, activation and residual), each with its
gradient as a ``*_backward`` call.

Names, defaults and streams only: the checks of the tensors, the allocation of
outputs and the calls into libep_gb300.so are in the compiled binding (_moe.so,
csrc/moe_binding.cpp), and every step runs in the library's CUDA kernels.  The
formulas are those of include/ep_api.h.  Every call is asynchronous on
``stream`` (default: the current one); what it allocates belongs to that
stream.  Inputs that another stream made have to be ready there, and to live
until the call's work is done (``Tensor.record_stream``).  Device-side problems
(an expert id out of range, a wait that gave up) set bits that ``moe_error``
reads.  The first call on a device creates its error word and may load device
code: make it before any stream capture.

Autograd does not follow these calls: whether or not an input requires a
gradient, the outputs do not, and the ``*_backward`` calls are the gradient (as
``examples/moe_layer.py`` chains them, or from a ``torch.autograd.Function``).
"""
from __future__ import annotations

import importlib.util
from typing import Optional, Sequence

import torch

from . import _lib
from . import build as _build


def _load_binding():
    _lib.load()                    # each is built if needed; raises if it cannot
    _build.build_binding()
    spec = importlib.util.spec_from_file_location("_moe", _build.BINDING)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.set_error_class(_lib.EpError)
    return module


_moe = _load_binding()


def _on(tensor, stream):
    """Context that makes ``stream`` current, on the tensors' device."""
    if not isinstance(tensor, torch.Tensor) or not tensor.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    if stream.device != tensor.device:
        raise ValueError("the stream is on another device than the tensors")
    return torch.cuda.stream(stream)


def moe_error(device=None) -> int:
    """Synchronise ``device`` and read and clear the EP_DEVERR_* bits that this
    module's calls set there."""
    index = torch.cuda.current_device() if device is None else torch.device(device).index
    if index is None:
        index = torch.cuda.current_device()
    torch.cuda.synchronize(index)
    t = _moe.error_word(index)
    bits = int(t.item())
    if bits:
        t.zero_()
        torch.cuda.synchronize(index)
    return bits


def route(logits: torch.Tensor, topk: int, *, score: str = "softmax", renormalize: bool = True,
          scale: float = 1.0, bias: Optional[torch.Tensor] = None,
          num_tokens: Optional[Sequence[int]] = None, stream=None):
    """Choose every token's ``topk`` experts and weigh them.

    logits: bf16, fp16 or fp32 [T][E] or [W][T][E] (rows may be strided).
    bias: fp32 [E], added to the logits, not to the scores, for the choice alone.
    (Where a load-balancing bias belongs to the score, as in sigmoid(x) + bias,
    ``route(torch.sigmoid(logits.float()), topk, bias=bias)`` chooses so, with
    -inf put back for closed experts, whose score is 0 otherwise; its indices go
    into ``route_backward`` with the logits as any others do.)  An expert whose
    logit is -inf or NaN is closed.  Returns (weights fp32, indices int32)
    [...][topk], as ``EpDispatchCombineOp.dispatch`` takes them; tokens
    t >= num_tokens[w] get weights 0 and indices -1."""
    if stream is not None:
        with _on(logits, stream):
            return _moe.route(logits, topk, score, renormalize, scale, bias, num_tokens)
    return _moe.route(logits, topk, score, renormalize, scale, bias, num_tokens)


def _backward(stream, logits, *args):
    if stream is not None:
        with _on(logits, stream):
            return _moe.route_backward(logits, *args)
    return _moe.route_backward(logits, *args)


def route_backward(grad_weights: torch.Tensor, logits: torch.Tensor, indices: torch.Tensor, *,
                   score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                   num_tokens: Optional[Sequence[int]] = None, grad_loss: Optional[torch.Tensor] = None,
                   counts: Optional[torch.Tensor] = None, balance_coef: float = 1.0, z_coef: float = 0.0,
                   stream=None) -> torch.Tensor:
    """Gradient of ``route``'s weights by the logits, dense and in their type.
    With grad_loss (one fp32 value) and counts, the gradient of
    ``balance_loss`` with these coefficients (its own defaults) is added in the
    same pass."""
    if grad_weights is None:
        raise ValueError("grad_weights is needed: balance_loss_backward is the loss's gradient alone")
    return _backward(stream, logits, indices.shape[-1], grad_weights, indices, grad_loss, counts, num_tokens,
                     score, renormalize, scale, balance_coef, z_coef)


def balance_loss(logits: torch.Tensor, indices: torch.Tensor, *, balance_coef: float = 1.0,
                 z_coef: float = 0.0, num_tokens: Optional[Sequence[int]] = None, stream=None):
    """Balance and z losses of a routing.  Returns (loss fp32 [3]: total,
    balance, z; counts int32 [E]: how often each expert was chosen; probs fp32
    [E]: mean router probability), over the tokens t < num_tokens[w]."""
    if stream is not None:
        with _on(logits, stream):
            return _moe.balance_loss(logits, indices, balance_coef, z_coef, num_tokens)
    return _moe.balance_loss(logits, indices, balance_coef, z_coef, num_tokens)


def balance_loss_backward(grad_loss: torch.Tensor, logits: torch.Tensor, counts: torch.Tensor, topk: int, *,
                          balance_coef: float = 1.0, z_coef: float = 0.0,
                          num_tokens: Optional[Sequence[int]] = None, stream=None) -> torch.Tensor:
    """Gradient of ``balance_loss``'s total by the logits; grad_loss is one
    fp32 value on the device, counts those that ``balance_loss`` returned."""
    return _backward(stream, logits, topk, None, None, grad_loss, counts, num_tokens,
                     "softmax", True, 1.0, balance_coef, z_coef)


def expert_product(x: torch.Tensor, weight: torch.Tensor, count: Optional[torch.Tensor] = None,
                   offset: Optional[torch.Tensor] = None, *, bias: Optional[torch.Tensor] = None,
                   activation: str = "none", residual: Optional[torch.Tensor] = None,
                   save_pre: bool = False, out: Optional[torch.Tensor] = None, stream=None):
    """y = act(x W_g^T + bias_g) + residual over the rows of every group g.

    x: bf16 or fp16 [rows][K] or [R][rows][K]; count, offset: int32 [R][G/R] as
    ``moe_group`` returns them (None: one group per rank holds all its rows);
    weight: [G][N][K]; activation "none", "relu", "gelu", "silu", or "swiglu"
    with weight [G][2N][K] (the gate's features first); bias: [G][weight's
    features].  residual and out: [...][N].  Returns y, or (y, pre) with
    save_pre: what ``expert_product_backward`` needs.  Rows outside every
    group are unspecified (untouched in ``out``).  out may be the residual
    itself and overlaps no other input."""
    if stream is not None:
        with _on(x, stream):
            return _moe.expert_product(x, weight, count, offset, bias, activation, residual, save_pre, out)
    return _moe.expert_product(x, weight, count, offset, bias, activation, residual, save_pre, out)


def expert_product_backward(grad: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                            count: Optional[torch.Tensor] = None, offset: Optional[torch.Tensor] = None, *,
                            pre: Optional[torch.Tensor] = None, activation: str = "none",
                            bias_grad: bool = False, stream=None):
    """Gradients of ``expert_product``: (grad_x, grad_weight, grad_bias or
    None) from grad = dL/dy.  pre: the forward's (not needed for "none").  The
    residual's gradient is grad itself.  Rows of grad_x outside every group
    are unspecified; a group without rows gets zero gradients."""
    if stream is not None:
        with _on(x, stream):
            return _moe.expert_product_backward(grad, x, weight, count, offset, pre, activation, bias_grad)
    return _moe.expert_product_backward(grad, x, weight, count, offset, pre, activation, bias_grad)
