"""What the routing, loss and product calls refuse: the C entry points on
arguments that the host can check (no GPU needed), and the Python face."""
import ctypes

import pytest
import torch

import combine_ep_layout_06_gb300 as ep
from combine_ep_layout_06_gb300 import _lib

INVALID = _lib.EP_ERR_INVALID_ARGS
P = ctypes.c_void_p(0x10000)               # never dereferenced: every call below is refused


@pytest.fixture(scope="module")
def L():
    return _lib.load()


def route_desc(**kw):
    d = dict(world_size=2, tokens=16, num_experts=64, topk=4, dtype=0, score=0, renormalize=1, scale=1.0,
             row_stride=64, rank_stride=1024)
    d.update(kw)
    return _lib.EpRouteDescC(**d)


BAD_ROUTE = [dict(world_size=0), dict(world_size=33), dict(tokens=0), dict(tokens=1 << 30), dict(num_experts=0),
             dict(num_experts=1025, row_stride=2000), dict(topk=0), dict(topk=33), dict(topk=5, num_experts=4),
             dict(dtype=1), dict(dtype=9), dict(score=2), dict(score=-1), dict(row_stride=63), dict(rank_stride=-1)]


@pytest.mark.parametrize("bad", BAD_ROUTE)
def test_route_descriptors(L, bad):
    d = ctypes.byref(route_desc(**bad))
    nt = (ctypes.c_int32 * 33)(*[1] * 33)
    n = ctypes.c_size_t(0)
    assert L.ep_route(d, P, None, nt, P, P, None) == INVALID
    assert L.ep_route_backward(d, P, P, P, None, None, nt, P, None, None) == INVALID
    assert L.ep_balance_loss_workspace(d, ctypes.byref(n)) == INVALID
    assert L.ep_balance_loss(d, P, P, nt, P, P, P, P, 1 << 30, None, None) == INVALID


def test_route_pointers_and_counts(L):
    d = ctypes.byref(route_desc())
    nt = (ctypes.c_int32 * 2)(16, 0)
    odd = ctypes.c_void_p(0x10001)
    assert L.ep_route(None, P, None, nt, P, P, None) == INVALID
    for i in (1, 3, 4, 5):
        a = [d, P, None, nt, P, P, None]
        a[i] = None
        assert L.ep_route(*a) == INVALID
    for i in (1, 2, 4, 5):
        a = [d, P, None, nt, P, P, None]
        a[i] = odd
        assert L.ep_route(*a) == INVALID
    for bad in ((17, 0), (-1, 3)):
        assert L.ep_route(d, P, None, (ctypes.c_int32 * 2)(*bad), P, P, None) == INVALID
    # halves of a pair, or nothing to differentiate
    for parts in ((P, None, None, None), (None, P, None, None), (None, None, P, None), (None, None, None, P), (None,) * 4):
        assert L.ep_route_backward(d, P, *parts, nt, P, None, None) == INVALID
    n = ctypes.c_size_t(0)
    assert L.ep_balance_loss_workspace(d, ctypes.byref(n)) == 0 and n.value > 0
    assert L.ep_balance_loss(d, P, P, nt, P, P, P, P, n.value - 1, None, None) == INVALID
    assert L.ep_balance_loss(d, P, P, nt, P, P, P, ctypes.c_void_p(0x10004), n.value, None, None) == INVALID


def rows(width=64, ptr=0x10000, rank=1 << 20):
    return _lib.EpRowsC(ptr, rank, width)


def product_desc(**kw):
    d = dict(ranks=2, groups=4, rows=100, in_features=64, out_features=32, dtype=0, activation=0, reserved=0,
             d_count=0x10000, d_offset=0x10000, weight=rows(), x=rows())
    d.update(kw)
    return _lib.EpProductDescC(**d)


BAD_PRODUCT = [dict(ranks=0), dict(groups=0), dict(groups=40000), dict(rows=-1), dict(rows=(1 << 30) + 1),
               dict(in_features=0), dict(in_features=60, weight=rows(), x=rows()), dict(out_features=0),
               dict(out_features=36), dict(out_features=(1 << 24) + 8), dict(dtype=2), dict(dtype=1), dict(activation=5),
               dict(activation=-1), dict(reserved=1), dict(d_count=None), dict(d_offset=None),
               dict(d_count=None, d_offset=None), dict(d_count=0x10002), dict(weight=rows(ptr=None)),
               dict(weight=rows(ptr=0x10008)), dict(weight=rows(56)), dict(weight=rows(68)), dict(weight=rows(rank=12)),
               dict(weight=rows(rank=-8)), dict(x=rows(ptr=0x10002)), dict(x=rows(56)), dict(x=rows(rank=4)),
               dict(x=rows(ptr=None))]


@pytest.mark.parametrize("bad", BAD_PRODUCT)
def test_product_descriptors(L, bad):
    d = ctypes.byref(product_desc(**bad))
    none, y = ctypes.byref(rows(ptr=None)), ctypes.byref(rows(32))
    n = ctypes.c_size_t(0)
    assert L.ep_expert_product(d, None, none, y, none, None, None) == INVALID
    assert L.ep_expert_product_workspace(d, ctypes.byref(n)) == INVALID
    assert L.ep_expert_product_backward(d, y, none, ctypes.byref(rows()), P, None, P, 1 << 40, None, None) == INVALID


def test_product_rows_and_workspace(L):
    none, y = rows(ptr=None), rows(32)
    ref = ctypes.byref
    good = ref(product_desc())
    for bad in (rows(ptr=None), rows(24), rows(36), rows(32, ptr=0x10004), rows(32, rank=3)):
        assert L.ep_expert_product(good, None, ref(none), ref(bad), ref(none), None, None) == INVALID
        if bad.ptr:
            assert L.ep_expert_product(good, None, ref(bad), ref(y), ref(none), None, None) == INVALID
            assert L.ep_expert_product(good, None, ref(none), ref(y), ref(bad), None, None) == INVALID
    assert L.ep_expert_product(good, None, None, ref(y), ref(none), None, None) == INVALID
    assert L.ep_expert_product(good, ctypes.c_void_p(0x10002), ref(none), ref(y), ref(none), None, None) == INVALID
    gated = ref(product_desc(activation=4))
    n = ctypes.c_size_t(0)
    assert L.ep_expert_product_workspace(gated, ref(n)) == 0 and n.value >= 2 * 100 * 64 * 2
    gx, pre = ref(rows()), ref(rows(64))
    assert L.ep_expert_product_backward(gated, ref(y), pre, gx, P, None, P, n.value - 1, None, None) == INVALID
    assert L.ep_expert_product_backward(gated, ref(y), pre, gx, P, None, None, n.value, None, None) == INVALID
    assert L.ep_expert_product_backward(gated, ref(y), ref(none), gx, P, None, P, n.value, None, None) == INVALID
    assert L.ep_expert_product_backward(gated, ref(y), ref(rows(32)), gx, P, None, P, n.value, None, None) == INVALID


def test_python_face_needs_gpu_tensors():
    x = torch.zeros((2, 4, 8))
    i = torch.zeros((2, 4, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        ep.route(x, 2)
    with pytest.raises(ValueError):
        ep.route_backward(torch.zeros((2, 4, 2)), x, i)
    with pytest.raises(ValueError):
        ep.balance_loss(x, i)
    with pytest.raises(ValueError):
        ep.balance_loss_backward(torch.zeros(()), x, torch.zeros(8, dtype=torch.int32), 2)
    h = torch.zeros((4, 16), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ep.expert_product(h, torch.zeros((1, 8, 16), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ep.expert_product_backward(h, h, torch.zeros((1, 16, 16), dtype=torch.bfloat16))


@pytest.mark.gpu
def test_python_face_refuses():
    c = "cuda"
    x = torch.zeros((2, 4, 8), device=c)
    i = torch.zeros((2, 4, 2), dtype=torch.int32, device=c)
    w = torch.zeros((2, 4, 2), device=c)
    counts = torch.zeros(8, dtype=torch.int32, device=c)
    one = torch.ones((), device=c)
    for call in (lambda: ep.route(x, 0), lambda: ep.route(x, 9), lambda: ep.route(x.double(), 2),
                 lambda: ep.route(x[0, 0], 2), lambda: ep.route(x, 2, score="linear"),
                 lambda: ep.route(x.transpose(1, 2), 2), lambda: ep.route(x, 2, num_tokens=[4]),
                 lambda: ep.route(x, 2, num_tokens=[5, 0]), lambda: ep.route(x, 2, num_tokens=[-1, 0]),
                 lambda: ep.route(x, 2, bias=torch.zeros(7, device=c)), lambda: ep.route(x, 2, bias=torch.zeros(8)),
                 lambda: ep.route(x[:, :1].expand(2, 4, 8), 2),
                 lambda: ep.route(torch.zeros((1, 1, 1025), device=c), 2),
                 lambda: ep.route_backward(w, x, i.long()), lambda: ep.route_backward(w.half(), x, i),
                 lambda: ep.route_backward(w[:1], x, i), lambda: ep.route_backward(w, x, i, grad_loss=one),
                 lambda: ep.route_backward(w, x, i, grad_loss=one, counts=counts[:4]),
                 lambda: ep.balance_loss(x, i[..., :1]), lambda: ep.balance_loss(x, i[:1]),
                 lambda: ep.balance_loss_backward(torch.ones(3, device=c), x, counts, 2),
                 lambda: ep.balance_loss_backward(None, x, counts, 2),
                 lambda: ep.balance_loss_backward(one, x, counts.float(), 2)):
        with pytest.raises(ValueError):
            call()
    h = torch.zeros((2, 6, 16), dtype=torch.bfloat16, device=c)
    wt = torch.zeros((4, 24, 16), dtype=torch.bfloat16, device=c)
    n = torch.zeros((2, 2), dtype=torch.int32, device=c)
    y = torch.zeros((2, 6, 24), dtype=torch.bfloat16, device=c)
    for call in (lambda: ep.expert_product(h.float(), wt.float(), n, n), lambda: ep.expert_product(h, wt.half(), n, n),
                 lambda: ep.expert_product(h, wt, n, None), lambda: ep.expert_product(h, wt),
                 lambda: ep.expert_product(h, wt, n.long(), n), lambda: ep.expert_product(h, wt, n[:1], n),
                 lambda: ep.expert_product(h, wt[:3], n, n), lambda: ep.expert_product(h, wt[:, :, :8], n, n),
                 lambda: ep.expert_product(h, wt[:, :20], n, n), lambda: ep.expert_product(h, wt, n, n, activation="tanh"),
                 lambda: ep.expert_product(h, wt, n, n, activation="swiglu"),
                 lambda: ep.expert_product(h, wt, n, n, bias=torch.zeros((4, 16), dtype=torch.bfloat16, device=c)),
                 lambda: ep.expert_product(h, wt, n, n, bias=torch.zeros((4, 24), device=c)),
                 lambda: ep.expert_product(h, wt, n, n, residual=h), lambda: ep.expert_product(h, wt, n, n, out=y[:, :5]),
                 lambda: ep.expert_product(h, wt, n, n, out=y.cpu()),
                 lambda: ep.expert_product(h.transpose(0, 1).contiguous().transpose(0, 1)[..., 1:9], wt[..., :8].contiguous(), n, n),
                 lambda: ep.expert_product_backward(y, h, wt, n, n, activation="silu"),
                 lambda: ep.expert_product_backward(h, h, wt, n, n)):
        with pytest.raises(ValueError):
            call()
    assert ep.moe_error() == 0
