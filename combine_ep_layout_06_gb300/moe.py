"""What stands before and between dispatch and combine in a MoE layer:
``route`` (router logits -> dispatch's weights and indices), ``balance_loss``
(the loss that evens out the experts' loads, with per-expert counts) and
``expert_product`` (one matrix product per expert over the rows that
``moe_group`` leaves, with bias, activation and residual), each with its
gradient as a ``*_backward`` call.

Marshalling only: every step runs in the CUDA kernels of libep_gb300.so.  The
formulas are those of include/ep_api.h.  Every call is asynchronous on
``stream`` (default: the current one); what it allocates belongs to that
stream.  Inputs that another stream made have to be ready there, and to live
until the call's work is done (``Tensor.record_stream``).  Device-side problems (an expert id out of range, a wait that gave up)
set bits that ``moe_error`` reads.  The first call on a device creates its
error word and may load device code: make it before any stream capture.

A single-token call takes a few microseconds on the GPU, so the host's part is
kept short: what shapes, strides and options alone decide is checked once and
remembered by their values (never by a tensor's address or identity), and C
descriptors are packed as bytes.
"""
from __future__ import annotations

import ctypes
import functools
import struct
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

# the descriptors' layouts (native alignment), as bytes
_ROUTE_DESC = struct.Struct("7i3f2q")
_ROWS = struct.Struct("Pqq")
_PRODUCT_HEAD = struct.Struct("8i")
_PRODUCT_TAIL = struct.Struct("PPPqqPqq")
assert _ROUTE_DESC.size == ctypes.sizeof(EpRouteDescC)
assert _ROWS.size == ctypes.sizeof(EpRowsC)
assert _PRODUCT_HEAD.size + _PRODUCT_TAIL.size == ctypes.sizeof(EpProductDescC)
_NO_ROWS = _ROWS.pack(0, 0, 0)

_lock = threading.Lock()
_error_words = {}                  # device index -> (the device's error word, its address)


def _error_word(index: int):
    t = _error_words.get(index)
    if t is None:
        with _lock:
            t = _error_words.get(index)
            if t is None:
                word = torch.zeros(1, dtype=torch.int32, device=torch.device("cuda", index))
                torch.cuda.current_stream(index).synchronize()   # zero for every stream
                t = _error_words[index] = (word, word.data_ptr())
    return t


def moe_error(device=None) -> int:
    """Synchronise ``device`` and read and clear the EP_DEVERR_* bits that this
    module's calls set there."""
    index = torch.cuda.current_device() if device is None else torch.device(device).index
    if index is None:
        index = torch.cuda.current_device()
    torch.cuda.synchronize(index)
    t = _error_word(index)[0]
    bits = int(t.item())
    if bits:
        t.zero_()
        torch.cuda.synchronize(index)
    return bits


@functools.lru_cache(maxsize=None)
def _entry(name: str):
    return getattr(_lib.load(), name)


# set once torch has CUDA; a machine without a GPU has only tensors to refuse
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _elsewhere(tensor, stream):
    """Context in which a call runs whose tensors' device is not the current
    one, or that names a stream: what it allocates and launches goes there."""
    if tensor is None or not tensor.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    if stream is None:
        return torch.cuda.device(tensor.get_device())
    if stream.device != tensor.device:
        raise ValueError("the stream is on another device than the tensors")
    return torch.cuda.stream(stream)


def _check_device(index, what, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"{what} must be on cuda:{index}")


# ------------------------------------------------------------ routing

@functools.lru_cache(maxsize=1024)
def _route_plan(shape, strides, dtype, topk, num_tokens, score, renormalize, scale, balance_coef, z_coef):
    """Descriptor, token counts, lead shape, T, E and the losses' scratch
    bytes for [T][E] or [W][T][E] logits."""
    if len(shape) not in (2, 3) or dtype not in _ROUTE_DTYPES:
        raise ValueError("logits must be bf16, fp16 or fp32 [T][E] or [W][T][E]")
    W, T, E = shape if len(shape) == 3 else (1, *shape)
    if not 1 <= E <= _lib.EP_MAX_ROUTE_EXPERTS:
        raise ValueError(f"1 to {_lib.EP_MAX_ROUTE_EXPERTS} experts, not {E}")
    if not 1 <= W <= _lib.EP_MAX_WORLD:
        raise ValueError(f"1 to {_lib.EP_MAX_WORLD} ranks, not {W}")
    if not 1 <= topk <= min(E, _lib.EP_MAX_TOPK):
        raise ValueError(f"topk must be 1 to {min(E, _lib.EP_MAX_TOPK)}, not {topk}")
    if score not in _SCORES:
        raise ValueError(f"score {score!r}: one of {sorted(_SCORES)}")
    if (strides[-1] != 1 and E > 1) or (strides[-2] < E and T > 1):
        raise ValueError("the rows of logits must be contiguous and must not overlap")
    if num_tokens is None:
        num_tokens = (T,) * W
    if len(num_tokens) != W or min(num_tokens) < 0 or max(num_tokens) > T:
        raise ValueError(f"num_tokens must be {W} counts of 0 to {T}")
    desc = _ROUTE_DESC.pack(W, T, E, topk, _ROUTE_DTYPES[dtype], _SCORES[score], int(bool(renormalize)),
                            scale, balance_coef, z_coef, max(strides[-2], E), strides[0] if W > 1 else 0)
    need = ctypes.c_size_t(0)
    if T:
        check(_entry("ep_balance_loss_workspace")(desc, ctypes.byref(need)), "ep_balance_loss_workspace")
    return desc, struct.pack(f"{W}i", *num_tokens), tuple(shape[:-1]), T, E, need.value


def _plan(logits, topk, num_tokens, score="softmax", renormalize=True, scale=1.0, balance_coef=0.0, z_coef=0.0):
    if num_tokens is not None:
        num_tokens = tuple(map(int, num_tokens))
    return _route_plan(logits.shape, logits.stride(), logits.dtype, topk, num_tokens, score, renormalize,
                       scale, balance_coef, z_coef)


def _dense(t, dtype, shape, name):
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
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
    index = logits.get_device()
    if stream is not None or index < 0 or index != _current_device():
        with _elsewhere(logits, stream):
            return route(logits, topk, score=score, renormalize=renormalize, scale=scale, bias=bias,
                         num_tokens=num_tokens)
    desc, counts, lead, T, E, _ = _plan(logits, topk, num_tokens, score, renormalize, scale)
    b = None
    if bias is not None:
        _check_device(index, "bias", bias)
        _dense(bias, torch.float32, (E,), "bias")
        b = bias.data_ptr()
    device = logits.device
    w = torch.empty((*lead, topk), dtype=torch.float32, device=device)
    idx = torch.empty((*lead, topk), dtype=torch.int32, device=device)
    if T:
        status = _entry("ep_route")(desc, logits.data_ptr(), b, counts, w.data_ptr(), idx.data_ptr(),
                                    _raw_stream(index))
        if status:
            check(status, "ep_route")
    return w, idx


def _backward(grad_weights, logits, indices, topk, grad_loss, loss_counts, num_tokens, stream, *options):
    index = logits.get_device()
    if stream is not None or index < 0 or index != _current_device():
        with _elsewhere(logits, stream):
            return _backward(grad_weights, logits, indices, topk, grad_loss, loss_counts, num_tokens, None, *options)
    desc, counts, lead, T, E, _ = _plan(logits, topk, num_tokens, *options)
    _check_device(index, "gradients, indices and counts", grad_weights, indices, grad_loss, loss_counts)
    gw = idx = gl = lc = None
    if grad_weights is not None:
        _dense(grad_weights, torch.float32, (*lead, topk), "grad_weights")
        _dense(indices, torch.int32, (*lead, topk), "indices")
        gw, idx = grad_weights.data_ptr(), indices.data_ptr()
    if grad_loss is not None:
        if loss_counts is None:
            raise ValueError("grad_loss needs the counts of balance_loss")
        if grad_loss.dtype != torch.float32 or grad_loss.numel() != 1:
            raise ValueError("grad_loss must be one fp32 value on the device")
        _dense(loss_counts, torch.int32, (E,), "counts")
        gl, lc = grad_loss.data_ptr(), loss_counts.data_ptr()
    out = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    if T:
        status = _entry("ep_route_backward")(desc, logits.data_ptr(), gw, idx, gl, lc, counts, out.data_ptr(),
                                             _error_word(index)[1], _raw_stream(index))
        if status:
            check(status, "ep_route_backward")
    return out


def route_backward(grad_weights: torch.Tensor, logits: torch.Tensor, indices: torch.Tensor, *,
                   score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                   num_tokens: Optional[Sequence[int]] = None, grad_loss: Optional[torch.Tensor] = None,
                   counts: Optional[torch.Tensor] = None, balance_coef: float = 0.0, z_coef: float = 0.0,
                   stream=None) -> torch.Tensor:
    """Gradient of ``route``'s weights by the logits, dense and in their type.
    With grad_loss (one fp32 value) and counts, the gradient of
    ``balance_loss`` with these coefficients is added in the same pass."""
    if grad_weights is None:
        raise ValueError("grad_weights is needed: balance_loss_backward is the loss's gradient alone")
    return _backward(grad_weights, logits, indices, indices.shape[-1], grad_loss, counts, num_tokens,
                     stream, score, renormalize, scale, balance_coef, z_coef)


def balance_loss(logits: torch.Tensor, indices: torch.Tensor, *, balance_coef: float = 1.0,
                 z_coef: float = 0.0, num_tokens: Optional[Sequence[int]] = None, stream=None):
    """Balance and z losses of a routing.  Returns (loss fp32 [3]: total,
    balance, z; counts int32 [E]: how often each expert was chosen; probs fp32
    [E]: mean router probability), over the tokens t < num_tokens[w]."""
    index = logits.get_device()
    if stream is not None or index < 0 or index != _current_device():
        with _elsewhere(logits, stream):
            return balance_loss(logits, indices, balance_coef=balance_coef, z_coef=z_coef, num_tokens=num_tokens)
    topk = indices.shape[-1]
    desc, nt, lead, T, E, need = _plan(logits, topk, num_tokens, "softmax", True, 1.0, balance_coef, z_coef)
    _check_device(index, "indices", indices)
    _dense(indices, torch.int32, (*lead, topk), "indices")
    device = logits.device
    loss = torch.empty(3, dtype=torch.float32, device=device)
    counts = torch.empty(E, dtype=torch.int32, device=device)
    probs = torch.empty(E, dtype=torch.float32, device=device)
    if T == 0:
        return loss.zero_(), counts.zero_(), probs.zero_()
    scratch = torch.empty(need, dtype=torch.uint8, device=device)
    status = _entry("ep_balance_loss")(desc, logits.data_ptr(), indices.data_ptr(), nt, loss.data_ptr(),
                                       counts.data_ptr(), probs.data_ptr(), scratch.data_ptr(), need,
                                       _error_word(index)[1], _raw_stream(index))
    if status:
        check(status, "ep_balance_loss")
    return loss, counts, probs


def balance_loss_backward(grad_loss: torch.Tensor, logits: torch.Tensor, counts: torch.Tensor, topk: int, *,
                          balance_coef: float = 1.0, z_coef: float = 0.0,
                          num_tokens: Optional[Sequence[int]] = None, stream=None) -> torch.Tensor:
    """Gradient of ``balance_loss``'s total by the logits; grad_loss is one
    fp32 value on the device, counts those that ``balance_loss`` returned."""
    if grad_loss is None:
        raise ValueError("grad_loss must be one fp32 value on the device")
    return _backward(None, logits, None, topk, grad_loss, counts, num_tokens, stream,
                     "softmax", True, 1.0, balance_coef, z_coef)


# ------------------------------------------------------------ products

@functools.lru_cache(maxsize=1024)
def _strides_of(shape, strides, name):
    """(rank stride, row stride) of rows that the kernels can read."""
    rank = strides[0] if len(strides) == 3 and shape[0] > 1 else 0
    row = strides[-2] if shape[-2] > 1 else -(-shape[-1] // 8) * 8
    if (strides[-1] != 1 or row < shape[-1] or (row | rank) % 8
            or (rank == 0 and len(strides) == 3 and shape[0] > 1)):
        raise ValueError(f"{name}: contiguous rows, with strides of a multiple of 8 elements")
    return rank, row


def _rows(t: torch.Tensor, dtype, lead, width: int, name: str) -> bytes:
    """A given [rows][width] or [R][rows][width] tensor."""
    shape = t.shape
    if t.dtype != dtype or shape[:-1] != lead or shape[-1] != width:
        raise ValueError(f"{name} must be {dtype} {[*lead, width]}")
    ptr = t.data_ptr()
    if ptr % 16:
        raise ValueError(f"{name} must be 16-byte aligned")
    return _ROWS.pack(ptr, *_strides_of(shape, t.stride(), name))


@functools.lru_cache(maxsize=1024)
def _product_plan(xshape, xstrides, wshape, wstrides, dtype, wdtype, activation, grouped):
    """The descriptor's head, the strides of weight and x, R's lead shape,
    rows, N, wide, groups, and the gradient's workspace bytes."""
    if dtype not in _PRODUCT_DTYPES or len(xshape) not in (2, 3):
        raise ValueError("x must be bf16 or fp16 [rows][K] or [R][rows][K]")
    R, rows, K = xshape if len(xshape) == 3 else (1, *xshape)
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation {activation!r}: one of {sorted(_ACTIVATIONS)}")
    if wdtype != dtype or len(wshape) != 3 or wshape[2] != K:
        raise ValueError(f"weight must be {dtype} [groups][features][{K}]")
    G, wide = wshape[0], wshape[1]
    N = wide // 2 if activation == "swiglu" else wide
    if K % 8 or K == 0 or N % 8 or N == 0 or (activation == "swiglu" and wide % 2):
        raise ValueError("feature counts must be multiples of 8")
    if R < 1 or G % R or G == 0:
        raise ValueError(f"{G} groups do not divide over {R} ranks")
    if not grouped and G != R:
        raise ValueError("without count and offset there is one group per rank")
    ws = _strides_of(wshape, wstrides, "weight")
    xs = _strides_of(xshape, xstrides, "x") if rows else (0, 0)
    head = _PRODUCT_HEAD.pack(R, G // R, rows, K, N, _PRODUCT_DTYPES[dtype], _ACTIVATIONS[activation], 0)
    # with pointers of the right kind: the size depends on the head alone
    some = 16 if grouped else 0
    need = ctypes.c_size_t(0)
    check(_entry("ep_expert_product_workspace")(head + _PRODUCT_TAIL.pack(some, some, 16, *ws, 16, *xs),
                                                ctypes.byref(need)), "ep_expert_product_workspace")
    return head, ws, xs, tuple(xshape[:-1]), rows, N, wide, G, need.value


def _product_desc(plan, index, x, weight, count, offset):
    head, ws, xs, _, rows, _, _, G, _ = plan
    c = o = 0
    if count is not None:
        _check_device(index, "weight, count and offset", weight, count, offset)
        if (count.dtype != torch.int32 or offset.dtype != torch.int32 or count.numel() != G or offset.numel() != G
                or not count.is_contiguous() or not offset.is_contiguous()):
            raise ValueError(f"count and offset must be contiguous int32 of {G} groups")
        c, o = count.data_ptr(), offset.data_ptr()
    else:
        _check_device(index, "weight", weight)
    w, p = weight.data_ptr(), x.data_ptr() if rows else 0
    if (w | p) % 16:
        raise ValueError("x and weight must be 16-byte aligned")
    return head + _PRODUCT_TAIL.pack(c, o, w, *ws, p, *xs)


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
    index = x.get_device()
    if stream is not None or index < 0 or index != _current_device():
        with _elsewhere(x, stream):
            return expert_product(x, weight, count, offset, bias=bias, activation=activation, residual=residual,
                                  save_pre=save_pre, out=out)
    if (count is None) != (offset is None):
        raise ValueError("count and offset come together")
    dtype = x.dtype
    plan = _product_plan(x.shape, x.stride(), weight.shape, weight.stride(), dtype, weight.dtype, activation,
                         count is not None)
    _, _, _, lead, rows, N, wide, G, _ = plan
    desc = _product_desc(plan, index, x, weight, count, offset)
    b, res, pre, p = None, _NO_ROWS, None, _NO_ROWS
    if bias is not None:
        _check_device(index, "bias", bias)
        _dense(bias, dtype, (G, wide), "bias")
        b = bias.data_ptr()
    if residual is not None:
        _check_device(index, "residual", residual)
        res = _rows(residual, dtype, lead, N, "residual")
    if out is None:
        y = torch.empty((*lead, N), dtype=dtype, device=x.device)
        o = _ROWS.pack(y.data_ptr(), rows * N, N)
    else:
        _check_device(index, "out", out)
        y, o = out, _rows(out, dtype, lead, N, "out")
    if save_pre:
        pre = torch.empty((*lead, wide), dtype=dtype, device=x.device)
        p = _ROWS.pack(pre.data_ptr(), rows * wide, wide)
    if rows:
        status = _entry("ep_expert_product")(desc, b, res, o, p, _error_word(index)[1], _raw_stream(index))
        if status:
            check(status, "ep_expert_product")
    return (y, pre) if save_pre else y


def expert_product_backward(grad: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                            count: Optional[torch.Tensor] = None, offset: Optional[torch.Tensor] = None, *,
                            pre: Optional[torch.Tensor] = None, activation: str = "none",
                            bias_grad: bool = False, stream=None):
    """Gradients of ``expert_product``: (grad_x, grad_weight, grad_bias or
    None) from grad = dL/dy.  pre: the forward's (not needed for "none").  The
    residual's gradient is grad itself.  Rows of grad_x outside every group
    are unspecified; a group without rows gets zero gradients."""
    index = x.get_device()
    if stream is not None or index < 0 or index != _current_device():
        with _elsewhere(x, stream):
            return expert_product_backward(grad, x, weight, count, offset, pre=pre, activation=activation,
                                           bias_grad=bias_grad)
    if (count is None) != (offset is None):
        raise ValueError("count and offset come together")
    dtype = x.dtype
    plan = _product_plan(x.shape, x.stride(), weight.shape, weight.stride(), dtype, weight.dtype, activation,
                         count is not None)
    _, _, _, lead, rows, N, wide, G, need = plan
    desc = _product_desc(plan, index, x, weight, count, offset)
    if pre is None and activation != "none":
        raise ValueError(f"the gradient of {activation!r} needs pre")
    _check_device(index, "grad and pre", grad, pre)
    g = _rows(grad, dtype, lead, N, "grad")
    p = _NO_ROWS if pre is None else _rows(pre, dtype, lead, wide, "pre")
    device, K = x.device, weight.shape[2]
    dx = torch.empty((*lead, K), dtype=dtype, device=device)
    dw = torch.empty((G, wide, K), dtype=dtype, device=device)
    db = torch.empty((G, wide), dtype=dtype, device=device) if bias_grad else None
    scratch = torch.empty(need, dtype=torch.uint8, device=device)
    status = _entry("ep_expert_product_backward")(
        desc, g, p, _ROWS.pack(dx.data_ptr(), rows * K, K), dw.data_ptr(), None if db is None else db.data_ptr(),
        scratch.data_ptr(), need, _error_word(index)[1], _raw_stream(index))
    if status:
        check(status, "ep_expert_product_backward")
    return dx, dw, db
