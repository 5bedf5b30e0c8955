"""What stands before and between dispatch and combine in a MoE layer:
``route`` (router logits -> dispatch's weights and indices), ``balance_loss``
(the loss that evens out the experts' loads, with per-expert counts) and
``expert_product`` (one matrix product per expert over the rows that
``moe_group`` leaves, with bias, activation and residual), each with its
gradient as a ``*_backward`` call.  Around them ``rms_norm`` (the norm before
the layer, in 8 bits where dispatch takes them so), ``checkpoint`` (activations
kept in 8 bits for the backward pass) and ``moe_few_tokens`` (the whole layer's
experts at decode).

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
                            pre: Optional[torch.Tensor] = None, pre_scales: Optional[torch.Tensor] = None,
                            activation: str = "none", bias_grad: bool = False, stream=None):
    """Gradients of ``expert_product``: (grad_x, grad_weight, grad_bias or
    None) from grad = dL/dy.  pre: the forward's (not needed for "none"), or its
    codes with pre_scales, as ``checkpoint`` keeps them.  The residual's
    gradient is grad itself.  Rows of grad_x outside every group
    are unspecified; a group without rows gets zero gradients."""
    if stream is not None:
        with _on(x, stream):
            return _moe.expert_product_backward(grad, x, weight, count, offset, pre, activation, bias_grad, pre_scales)
    return _moe.expert_product_backward(grad, x, weight, count, offset, pre, activation, bias_grad, pre_scales)


def checkpoint(x: torch.Tensor, count: Optional[torch.Tensor] = None, offset: Optional[torch.Tensor] = None, *,
               stream=None):
    """Keep activations in 8 bits until the backward pass: (codes float8_e4m3fn,
    scales fp32 [...][ceil(F / 128)]) of the rows x [rows][F] or [R][rows][F], bf16
    or fp16, in every group (count, offset as for ``expert_product``).  One scale
    for every 128 values of a row, as dispatch quantises; a block with an infinity
    or a NaN is NaN as a whole.  Rows outside every group are unspecified."""
    if stream is not None:
        with _on(x, stream):
            return _moe.checkpoint(x, count, offset)
    return _moe.checkpoint(x, count, offset)


def checkpoint_restore(codes: torch.Tensor, scales: torch.Tensor, count: Optional[torch.Tensor] = None,
                       offset: Optional[torch.Tensor] = None, *, activation: str = "none",
                       dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """act(code * scale) of the rows of every group, bf16 or fp16: what was kept
    (activation "none"), or the activations of kept pre-activations, recomputed
    ("swiglu": half as many features).  codes: float8_e4m3fn or uint8, so the
    grouped rows of an FP8 dispatch as well."""
    if dtype not in _CODES:
        raise ValueError("dtype must be torch.bfloat16 or torch.float16")
    if stream is not None:
        with _on(codes, stream):
            return _moe.checkpoint_restore(codes, scales, count, offset, activation, _CODES[dtype])
    return _moe.checkpoint_restore(codes, scales, count, offset, activation, _CODES[dtype])


_CODES = {torch.bfloat16: _lib.EP_DT_BF16, torch.float16: _lib.EP_DT_FP16}


def rms_norm(x: torch.Tensor, weight: torch.Tensor, *, residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
             quantize: bool = False, stream=None):
    """y = total / sqrt(mean(total^2) + eps) * weight, total = x + residual.

    x: bf16, fp16 or fp32 [...][H], H to 32768; weight [H] in x's type or fp32.
    Returns y; with a residual (y, total), total rounded to x's type, whose norm
    it is.  eps: 0 or more (with 0, rows of a root mean square of 2^-127 or more).
    quantize: in y's place codes (float8_e4m3fn) and scales (fp32
    [...][H/128]), H a multiple of 128: ``EpDispatchCombineOp.dispatch`` takes
    them as pre-quantised input."""
    if stream is not None:
        with _on(x, stream):
            return _moe.rms_norm(x, weight, residual, eps, quantize)
    return _moe.rms_norm(x, weight, residual, eps, quantize)


def rms_norm_backward(grad: torch.Tensor, total: torch.Tensor, weight: torch.Tensor, *,
                      grad_total: Optional[torch.Tensor] = None, eps: float = 1e-6, stream=None):
    """Gradients of ``rms_norm`` from grad = dL/dy: (grad_x, grad_weight).
    total: the forward's, or x where there was no residual.  grad_total: what
    reaches total by other ways, added.  grad_x is the residual's gradient too."""
    if stream is not None:
        with _on(total, stream):
            return _moe.rms_norm_backward(grad, total, weight, grad_total, eps)
    return _moe.rms_norm_backward(grad, total, weight, grad_total, eps)


def moe_few_tokens(x: torch.Tensor, weights: torch.Tensor, indices: torch.Tensor, up: torch.Tensor,
                   down: torch.Tensor, *, activation: str = "swiglu", up_bias: Optional[torch.Tensor] = None,
                   down_bias: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """The experts of at most 64 tokens, without dispatch: out[t] = residual[t] +
    sum over j of weights[t][j] * y(t, indices[t][j]), y(t, e) = act(x[t] up[e]^T
    + up_bias[e]) down[e]^T + down_bias[e].

    x, residual: bf16 or fp16 [T][H] or [W][T][H]; weights fp32 and indices int32
    [...][topk] as ``route`` returns them (a negative index: no expert, so absent tokens
    get their residual or 0); up: [E][F][H], or [E][2F][H] for "swiglu" (the
    gate's features first); down: [E][H][F].  Sums are fp32, out is rounded once.
    fp16 activations between the products hold values up to 2^20 where the weights
    over all choices are more than 48 MB, and all of fp32's below."""
    if stream is not None:
        with _on(x, stream):
            return _moe.moe_few_tokens(x, weights, indices, up, down, activation, up_bias, down_bias, residual)
    return _moe.moe_few_tokens(x, weights, indices, up, down, activation, up_bias, down_bias, residual)
