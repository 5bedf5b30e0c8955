"""What stands before and between dispatch and combine in a MoE layer:
``route`` (router logits -> dispatch's weights and indices), ``balance_loss``
(the loss that evens out the experts' loads, with per-expert counts) and
``expert_product`` (one matrix product per expert over the rows that
``moe_group`` leaves, with bias, activation and residual), each with its
gradient as a ``*_backward`` call.

Marshalling only: every step runs in the CUDA kernels of libep_gb300.so.  The
formulas are those of include/ep_api.h.  Every call is asynchronous on
``stream`` (default: the current one); what it allocates belongs to that
stream.  Device-side problems (an expert id out of range, a wait that gave up)
set bits that ``moe_error`` reads.
"""
from __future__ import annotations

import ctypes
import threading
from typing import Optional, Sequence

import torch

from . import _lib
from ._lib import EpProductDescC, EpRouteDescC, EpRowsC, check

_ROUTE_DTYPES = {torch.bfloat16: _lib.EP_DT_BF16, torch.float16: _lib.EP_DT_FP16,
                 torch.float32: _lib.EP_DT_FP32}
_PRODUCT_DTYPES = {torch.bfloat16: _lib.EP_DT_BF16, torch.float16: _lib.EP_DT_FP16}
_SCORES = {"softmax": 0, "sigmoid": 1}
_ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3, "swiglu": 4}

_lock = threading.Lock()
_error_words = {}                  # device index -> the device's error word


def _error_word(index: int) -> torch.Tensor:
    t = _error_words.get(index)
    if t is None:
        with _lock:
            t = _error_words.get(index)
            if t is None:
                t = torch.zeros(1, dtype=torch.int32, device=torch.device("cuda", index))
                torch.cuda.current_stream(index).synchronize()   # zero for every stream
                _error_words[index] = t
    return t


def moe_error(device=None) -> int:
    """Synchronise ``device`` and read and clear the EP_DEVERR_* bits that this
    module's calls set there."""
    index = torch.cuda.current_device() if device is None else torch.device(device).index
    if index is None:
        index = torch.cuda.current_device()
    torch.cuda.synchronize(index)
    t = _error_word(index)
    bits = int(t.item())
    if bits:
        t.zero_()
        torch.cuda.synchronize(index)
    return bits


class _On:
    """Makes the tensors' device and the call's stream current."""

    def __init__(self, device, stream):
        if stream is not None and stream.device != device:
            raise ValueError("the stream is on another device than the tensors")
        self.guard = None
        if stream is not None:
            self.guard = torch.cuda.stream(stream)
        elif torch.cuda.current_device() != device.index:
            self.guard = torch.cuda.device(device)
        self.index = device.index

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return torch.cuda.current_stream(self.index).cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _on_gpu(t: torch.Tensor, what: str):
    if not t.is_cuda:
        raise ValueError(f"{what} must be on a CUDA device")


def _same_device(like: torch.Tensor, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != like.device:
            raise ValueError(f"{name} must be on {like.device}")


# ------------------------------------------------------------ routing

def _route_desc(logits, topk, num_tokens, score="softmax", renormalize=True, scale=1.0,
                balance_coef=0.0, z_coef=0.0):
    """Descriptor, token counts, and the (W, T) that a [T][E] or [W][T][E]
    tensor of logits stands for."""
    _on_gpu(logits, "logits")
    if logits.dim() not in (2, 3) or logits.dtype not in _ROUTE_DTYPES:
        raise ValueError("logits must be bf16, fp16 or fp32 [T][E] or [W][T][E]")
    shape = tuple(logits.shape)
    W, T, E = shape if len(shape) == 3 else (1, *shape)
    if not 1 <= E <= _lib.EP_MAX_ROUTE_EXPERTS:
        raise ValueError(f"1 to {_lib.EP_MAX_ROUTE_EXPERTS} experts, not {E}")
    if not 1 <= W <= _lib.EP_MAX_WORLD:
        raise ValueError(f"1 to {_lib.EP_MAX_WORLD} ranks, not {W}")
    if not 1 <= topk <= min(E, _lib.EP_MAX_TOPK):
        raise ValueError(f"topk must be 1 to {min(E, _lib.EP_MAX_TOPK)}, not {topk}")
    if score not in _SCORES:
        raise ValueError(f"score {score!r}: one of {sorted(_SCORES)}")
    strides = logits.stride()
    if (strides[-1] != 1 and E > 1) or (strides[-2] < E and T > 1):
        raise ValueError("the rows of logits must be contiguous and must not overlap")
    if num_tokens is None:
        counts = [T] * W
    else:
        counts = [int(n) for n in num_tokens]
        if len(counts) != W or min(counts) < 0 or max(counts) > T:
            raise ValueError(f"num_tokens must be {W} counts of 0 to {T}")
    desc = EpRouteDescC(W, T, E, topk, _ROUTE_DTYPES[logits.dtype], _SCORES[score], int(bool(renormalize)),
                        scale, balance_coef, z_coef, max(strides[-2], E), strides[0] if W > 1 else 0)
    return desc, (ctypes.c_int32 * W)(*counts), W, T, E


def _dense(t, dtype, shape, name):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {list(shape)}")


def route(logits: torch.Tensor, topk: int, *, score: str = "softmax", renormalize: bool = True,
          scale: float = 1.0, bias: Optional[torch.Tensor] = None,
          num_tokens: Optional[Sequence[int]] = None, stream=None):
    """Choose every token's ``topk`` experts and weigh them.

    logits: bf16, fp16 or fp32 [T][E] or [W][T][E] (rows may be strided).
    bias: fp32 [E], added to the logits for the choice alone.  An expert whose
    logit is -inf or NaN is closed.  Returns (weights fp32, indices int32)
    [...][topk], as ``EpDispatchCombineOp.dispatch`` takes them; tokens
    t >= num_tokens[w] get weights 0 and indices -1."""
    desc, counts, W, T, E = _route_desc(logits, topk, num_tokens, score, renormalize, scale)
    if bias is not None:
        _same_device(logits, bias=bias)
        _dense(bias, torch.float32, (E,), "bias")
    lead = logits.shape[:-1]
    with _On(logits.device, stream) as st:
        w = torch.empty((*lead, topk), dtype=torch.float32, device=logits.device)
        idx = torch.empty((*lead, topk), dtype=torch.int32, device=logits.device)
        if T == 0:
            return w, idx
        check(_lib.load().ep_route(ctypes.byref(desc), logits.data_ptr(),
                                   None if bias is None else bias.data_ptr(), counts, w.data_ptr(),
                                   idx.data_ptr(), st), "ep_route")
    return w, idx


def _backward(grad_weights, logits, indices, topk, grad_loss, counts, num_tokens, stream, **options):
    desc, nt, W, T, E = _route_desc(logits, topk, num_tokens, **options)
    _same_device(logits, grad_weights=grad_weights, indices=indices, grad_loss=grad_loss, counts=counts)
    lead = logits.shape[:-1]
    if grad_weights is not None:
        _dense(grad_weights, torch.float32, (*lead, topk), "grad_weights")
        _dense(indices, torch.int32, (*lead, topk), "indices")
    if grad_loss is not None:
        if counts is None:
            raise ValueError("grad_loss needs the counts of balance_loss")
        if grad_loss.dtype != torch.float32 or grad_loss.numel() != 1:
            raise ValueError("grad_loss must be one fp32 value on the device")
        _dense(counts, torch.int32, (E,), "counts")
    with _On(logits.device, stream) as st:
        out = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        if T == 0:
            return out
        check(_lib.load().ep_route_backward(
            ctypes.byref(desc), logits.data_ptr(),
            None if grad_weights is None else grad_weights.data_ptr(),
            None if grad_weights is None else indices.data_ptr(),
            None if grad_loss is None else grad_loss.data_ptr(),
            None if grad_loss is None else counts.data_ptr(), nt, out.data_ptr(),
            _error_word(logits.device.index).data_ptr(), st), "ep_route_backward")
    return out


def route_backward(grad_weights: torch.Tensor, logits: torch.Tensor, indices: torch.Tensor, *,
                   score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                   num_tokens: Optional[Sequence[int]] = None, grad_loss: Optional[torch.Tensor] = None,
                   counts: Optional[torch.Tensor] = None, balance_coef: float = 0.0, z_coef: float = 0.0,
                   stream=None) -> torch.Tensor:
    """Gradient of ``route``'s weights by the logits, dense and in their type.
    With grad_loss (one fp32 value) and counts, the gradient of
    ``balance_loss`` with these coefficients is added in the same pass."""
    return _backward(grad_weights, logits, indices, indices.shape[-1], grad_loss, counts, num_tokens,
                     stream, score=score, renormalize=renormalize, scale=scale,
                     balance_coef=balance_coef, z_coef=z_coef)


def balance_loss(logits: torch.Tensor, indices: torch.Tensor, *, balance_coef: float = 1.0,
                 z_coef: float = 0.0, num_tokens: Optional[Sequence[int]] = None, stream=None):
    """Balance and z losses of a routing.  Returns (loss fp32 [3]: total,
    balance, z; counts int32 [E]: how often each expert was chosen; probs fp32
    [E]: mean router probability), over the tokens t < num_tokens[w]."""
    topk = indices.shape[-1]
    desc, nt, W, T, E = _route_desc(logits, topk, num_tokens, balance_coef=balance_coef, z_coef=z_coef)
    _same_device(logits, indices=indices)
    _dense(indices, torch.int32, (*logits.shape[:-1], topk), "indices")
    L = _lib.load()
    dev = logits.device
    with _On(dev, stream) as st:
        loss = torch.empty(3, dtype=torch.float32, device=dev)
        counts = torch.empty(E, dtype=torch.int32, device=dev)
        probs = torch.empty(E, dtype=torch.float32, device=dev)
        if T == 0:
            return loss.zero_(), counts.zero_(), probs.zero_()
        need = ctypes.c_size_t(0)
        check(L.ep_balance_loss_workspace(ctypes.byref(desc), ctypes.byref(need)), "ep_balance_loss_workspace")
        scratch = torch.empty(need.value, dtype=torch.uint8, device=dev)
        check(L.ep_balance_loss(ctypes.byref(desc), logits.data_ptr(), indices.data_ptr(), nt,
                                loss.data_ptr(), counts.data_ptr(), probs.data_ptr(), scratch.data_ptr(),
                                need.value, _error_word(dev.index).data_ptr(), st), "ep_balance_loss")
    return loss, counts, probs


def balance_loss_backward(grad_loss: torch.Tensor, logits: torch.Tensor, counts: torch.Tensor, topk: int, *,
                          balance_coef: float = 1.0, z_coef: float = 0.0,
                          num_tokens: Optional[Sequence[int]] = None, stream=None) -> torch.Tensor:
    """Gradient of ``balance_loss``'s total by the logits; grad_loss is one
    fp32 value on the device, counts those that ``balance_loss`` returned."""
    if grad_loss is None:
        raise ValueError("grad_loss must be one fp32 value on the device")
    return _backward(None, logits, None, topk, grad_loss, counts, num_tokens, stream,
                     balance_coef=balance_coef, z_coef=z_coef)


# ------------------------------------------------------------ products

def _rows(t: Optional[torch.Tensor], like, width: int, name: str) -> EpRowsC:
    """A [rows][width] or [R][rows][width] tensor of x's type and rows."""
    if t is None:
        return EpRowsC(None, 0, 0)
    shape = tuple(t.shape)
    if t.dtype != like.dtype or shape[:-1] != tuple(like.shape[:-1]) or shape[-1] != width:
        raise ValueError(f"{name} must be {like.dtype} {[*like.shape[:-1], width]}")
    return _strided(t, name)


def _strided(t: torch.Tensor, name: str) -> EpRowsC:
    strides = t.stride()
    rank = strides[0] if len(strides) == 3 and t.shape[0] > 1 else 0
    row = strides[-2] if t.shape[-2] > 1 else -(-t.shape[-1] // 8) * 8
    if (strides[-1] != 1 or row < t.shape[-1] or (row | rank) % 8 or t.data_ptr() % 16
            or (rank == 0 and len(strides) == 3 and t.shape[0] > 1)):
        raise ValueError(f"{name}: contiguous rows, 16-byte aligned, with strides of a multiple of 8 elements")
    return EpRowsC(t.data_ptr(), rank, row)


def _product_desc(x, weight, count, offset, activation):
    _on_gpu(x, "x")
    if x.dtype not in _PRODUCT_DTYPES or x.dim() not in (2, 3):
        raise ValueError("x must be bf16 or fp16 [rows][K] or [R][rows][K]")
    shape = tuple(x.shape)
    R, rows, K = shape if len(shape) == 3 else (1, *shape)
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation {activation!r}: one of {sorted(_ACTIVATIONS)}")
    if weight.dtype != x.dtype or weight.dim() != 3 or weight.shape[2] != K:
        raise ValueError(f"weight must be {x.dtype} [groups][features][{K}]")
    G, wide = weight.shape[0], weight.shape[1]
    N = wide // 2 if activation == "swiglu" else wide
    if K % 8 or K == 0 or N % 8 or N == 0 or (activation == "swiglu" and wide % 2):
        raise ValueError("feature counts must be multiples of 8")
    if R < 1 or G % R or G == 0:
        raise ValueError(f"{G} groups do not divide over {R} ranks")
    _same_device(x, weight=weight, count=count, offset=offset)
    if (count is None) != (offset is None):
        raise ValueError("count and offset come together")
    if count is None:
        if G != R:
            raise ValueError("without count and offset there is one group per rank")
    else:
        for name, t in (("count", count), ("offset", offset)):
            if t.dtype != torch.int32 or t.numel() != G or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous int32 [{R}][{G // R}]")
    desc = EpProductDescC(R, G // R, rows, K, N, _PRODUCT_DTYPES[x.dtype], _ACTIVATIONS[activation], 0,
                          None if count is None else count.data_ptr(),
                          None if offset is None else offset.data_ptr(),
                          _strided(weight, "weight"), _strided(x, "x") if rows else EpRowsC(None, 0, 0))
    return desc, N, wide


def _bias(bias, x, G, wide):
    if bias is None:
        return None
    _same_device(x, bias=bias)
    _dense(bias, x.dtype, (G, wide), "bias")
    return bias.data_ptr()


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
    group are unspecified (untouched in ``out``)."""
    desc, N, wide = _product_desc(x, weight, count, offset, activation)
    _same_device(x, residual=residual, out=out)
    b = _bias(bias, x, weight.shape[0], wide)
    res = _rows(residual, x, N, "residual")
    lead = x.shape[:-1]
    with _On(x.device, stream) as st:
        y = torch.empty((*lead, N), dtype=x.dtype, device=x.device) if out is None else out
        pre = torch.empty((*lead, wide), dtype=x.dtype, device=x.device) if save_pre else None
        if desc.rows:
            check(_lib.load().ep_expert_product(
                ctypes.byref(desc), b, ctypes.byref(res), ctypes.byref(_rows(y, x, N, "out")),
                ctypes.byref(_rows(pre, x, wide, "pre")), _error_word(x.device.index).data_ptr(), st),
                "ep_expert_product")
    return (y, pre) if save_pre else y


def expert_product_backward(grad: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                            count: Optional[torch.Tensor] = None, offset: Optional[torch.Tensor] = None, *,
                            pre: Optional[torch.Tensor] = None, activation: str = "none",
                            bias_grad: bool = False, stream=None):
    """Gradients of ``expert_product``: (grad_x, grad_weight, grad_bias or
    None) from grad = dL/dy.  pre: the forward's (not needed for "none").  The
    residual's gradient is grad itself.  Rows of grad_x outside every group
    are unspecified; a group without rows gets zero gradients."""
    desc, N, wide = _product_desc(x, weight, count, offset, activation)
    _same_device(x, grad=grad, pre=pre)
    if pre is None and activation != "none":
        raise ValueError(f"the gradient of {activation!r} needs pre")
    g = _rows(grad, x, N, "grad")
    p = _rows(pre, x, wide, "pre")
    L = _lib.load()
    with _On(x.device, stream) as st:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dw = torch.empty(weight.shape, dtype=x.dtype, device=x.device)
        db = torch.empty((weight.shape[0], wide), dtype=x.dtype, device=x.device) if bias_grad else None
        need = ctypes.c_size_t(0)
        check(L.ep_expert_product_workspace(ctypes.byref(desc), ctypes.byref(need)), "ep_expert_product_workspace")
        scratch = torch.empty(need.value, dtype=torch.uint8, device=x.device)
        check(L.ep_expert_product_backward(
            ctypes.byref(desc), ctypes.byref(g), ctypes.byref(p), ctypes.byref(_rows(dx, x, x.shape[-1], "x")),
            dw.data_ptr(), None if db is None else db.data_ptr(), scratch.data_ptr(), need.value,
            _error_word(x.device.index).data_ptr(), st), "ep_expert_product_backward")
    return dx, dw, db
