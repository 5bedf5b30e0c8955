"""What the norm, checkpoint and few-token calls refuse, without a GPU: the C
entry points check everything before their first CUDA call."""
import ctypes
import math

import pytest
import torch

import combine_ep_layout_06_gb300 as ep
from combine_ep_layout_06_gb300 import _lib, build

INVALID = _lib.EP_ERR_INVALID_ARGS
P = ctypes.c_void_p(0x10000)
ref = ctypes.byref


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.load()


def rows(width=64, ptr=0x10000, rank=1 << 20):
    return _lib.EpRowsC(ptr, rank, width)


NONE = rows(ptr=None)


def norm(**kw):
    d = dict(ranks=2, rows=8, width=256, dtype=0, weight_dtype=0, eps=1e-6, x=rows(256), weight=0x10000)
    d.update(kw)
    return _lib.EpNormDescC(**d)


@pytest.mark.parametrize("bad", [
    dict(ranks=0), dict(ranks=65536), dict(rows=-1), dict(rows=1 << 30), dict(width=0), dict(width=32769), dict(dtype=1), dict(dtype=4),
    dict(weight_dtype=3), dict(weight_dtype=1), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(weight=None), dict(weight=0x10001),
    dict(x=NONE), dict(x=rows(255)), dict(x=rows(256, ptr=0x10001)), dict(x=rows(256, rank=0))])
def test_norm_descriptors(L, bad):
    n = ctypes.c_size_t(0)
    d = ref(norm(**bad))
    assert L.ep_rms_norm(d, ref(NONE), ref(NONE), ref(rows(256)), ref(NONE), None) == INVALID
    assert L.ep_rms_norm_workspace(d, ref(n)) == INVALID
    assert L.ep_rms_norm_backward(d, ref(rows(256)), ref(NONE), ref(rows(256)), P, P, 1 << 40, None, None) == INVALID


def test_norm_rows(L):
    d, y, none = ref(norm()), ref(rows(256)), ref(NONE)
    for bad in (rows(255), rows(256, ptr=0x10001), rows(256, rank=-1)):
        for at in range(3):
            a = [none, none, y]
            a[at] = ref(bad)
            assert L.ep_rms_norm(d, *a, none, None) == INVALID
    assert L.ep_rms_norm(d, none, none, none, none, None) == INVALID
    assert L.ep_rms_norm(None, none, none, y, none, None) == INVALID
    for at in range(4):
        a = [none, none, y, none]
        a[at] = None
        assert L.ep_rms_norm(d, *a, None) == INVALID
    # codes: whole blocks, and scales' rows
    assert L.ep_rms_norm(ref(norm(width=200)), none, none, y, ref(rows(2)), None) == INVALID
    for bad in (rows(1), rows(2, ptr=0x10002), rows(2, rank=0)):
        assert L.ep_rms_norm(d, none, none, y, ref(bad), None) == INVALID
    n = ctypes.c_size_t(0)
    assert L.ep_rms_norm_workspace(d, ref(n)) == 0 and n.value >= 256 * 4
    for a in ([ref(rows(255)), none, y, P, P, n.value], [y, ref(rows(255)), y, P, P, n.value], [y, none, ref(rows(255)), P, P, n.value],
              [y, none, y, None, P, n.value], [y, none, y, P, None, n.value], [y, none, y, P, P, n.value - 1],
              [y, none, y, ctypes.c_void_p(0x10001), P, n.value], [y, none, y, P, ctypes.c_void_p(0x10004), n.value]):
        assert L.ep_rms_norm_backward(d, *a, None, None) == INVALID
    assert L.ep_rms_norm_backward(d, y, none, y, P, P, n.value, ctypes.c_void_p(0x10002), None) == INVALID
    assert L.ep_rms_norm(ref(norm(rows=0, x=NONE)), none, none, none, none, None) == 0


def checkpoint(**kw):
    d = dict(ranks=2, groups=4, rows=100, features=64, dtype=0, activation=0, d_count=0x10000, d_offset=0x10000)
    d.update(kw)
    return _lib.EpCheckpointDescC(**d)


@pytest.mark.parametrize("bad", [
    dict(ranks=0), dict(groups=0), dict(groups=40000), dict(rows=-1), dict(rows=(1 << 30) + 1), dict(features=0), dict(features=60),
    dict(features=(1 << 24) + 8), dict(dtype=1), dict(dtype=2), dict(activation=5), dict(activation=-1), dict(d_count=None),
    dict(d_offset=None), dict(d_count=None, d_offset=None), dict(d_count=0x10002)])
def test_checkpoint_descriptors(L, bad):
    d = ref(checkpoint(**bad))
    assert L.ep_checkpoint_save(d, ref(rows()), ref(rows()), ref(rows(1)), None) == INVALID
    assert L.ep_checkpoint_restore(d, ref(rows()), ref(rows(1)), ref(rows()), None) == INVALID


def test_checkpoint_rows(L):
    d, x, q, s = ref(checkpoint()), rows(), rows(), rows(1)
    for bad in (NONE, rows(56), rows(68), rows(ptr=0x10004), rows(rank=-8), rows(rank=4)):
        assert L.ep_checkpoint_save(d, ref(bad), ref(q), ref(s), None) == INVALID
        assert L.ep_checkpoint_save(d, ref(x), ref(bad), ref(s), None) == INVALID
        assert L.ep_checkpoint_restore(d, ref(bad), ref(s), ref(x), None) == INVALID
        assert L.ep_checkpoint_restore(d, ref(q), ref(s), ref(bad), None) == INVALID
    for bad in (NONE, rows(0), rows(1, ptr=0x10002), rows(1, rank=0)):
        assert L.ep_checkpoint_save(d, ref(x), ref(q), ref(bad), None) == INVALID
        assert L.ep_checkpoint_restore(d, ref(q), ref(bad), ref(x), None) == INVALID
    assert L.ep_checkpoint_restore(ref(checkpoint(features=72, activation=4)), ref(rows(72)), ref(s), ref(rows(72)), None) == INVALID
    for at in range(3):
        a = [ref(x), ref(q), ref(s)]
        a[at] = None
        assert L.ep_checkpoint_save(d, *a, None) == INVALID
        assert L.ep_checkpoint_restore(d, *a, None) == INVALID
    assert L.ep_checkpoint_save(ref(checkpoint(rows=0)), ref(NONE), ref(NONE), ref(NONE), None) == 0


def test_product_gradient_from_codes(L):
    p = _lib.EpProductDescC(ranks=2, groups=4, rows=100, in_features=64, out_features=32, dtype=0, activation=4, reserved=0,
                            d_count=0x10000, d_offset=0x10000, weight=rows(), x=rows())
    n = ctypes.c_size_t(0)
    assert L.ep_expert_product_workspace(ref(p), ref(n)) == 0
    for q, s in ((NONE, rows(1)), (rows(56), rows(1)), (rows(), NONE), (rows(), rows(1, ptr=0x10001)), (rows(ptr=0x10004), rows(1))):
        assert L.ep_expert_product_backward_checkpoint(ref(p), ref(rows(32)), ref(q), ref(s), ref(rows()), P, None, P, n.value, None,
                                                       None) == INVALID
    assert L.ep_expert_product_backward_checkpoint(ref(p), ref(rows(32)), ref(rows()), None, ref(rows()), P, None, P, n.value, None,
                                                   None) == INVALID


def few(**kw):
    d = dict(tokens=4, experts=8, topk=2, hidden=64, inner=32, dtype=0, activation=4, reserved=0, up=rows(), down=rows(32),
             up_bias=None, down_bias=None)
    d.update(kw)
    return _lib.EpFewDescC(**d)


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(tokens=65), dict(experts=0), dict(experts=1025), dict(topk=0), dict(topk=33), dict(hidden=0), dict(hidden=60),
    dict(hidden=(1 << 20) + 8), dict(inner=0), dict(inner=36), dict(inner=(1 << 20) + 8), dict(dtype=2), dict(dtype=1), dict(activation=5),
    dict(activation=-1), dict(reserved=1), dict(up=NONE), dict(up=rows(56)), dict(up=rows(68)), dict(up=rows(rank=0)), dict(up=rows(ptr=0x10008)),
    dict(down=rows(24)), dict(down=NONE), dict(up_bias=0x10002), dict(down_bias=0x10008)])
def test_few_descriptors(L, bad):
    n = ctypes.c_size_t(0)
    d = ref(few(**bad))
    assert L.ep_moe_few_workspace(d, ref(n)) == INVALID
    assert L.ep_moe_few(d, ref(rows()), P, P, ref(NONE), ref(rows()), P, 1 << 40, None, None) == INVALID


def test_few_rows(L):
    d, n = ref(few()), ctypes.c_size_t(0)
    assert L.ep_moe_few_workspace(d, ref(n)) == 0 and n.value > 0
    good = [ref(rows()), P, P, ref(NONE), ref(rows()), P, n.value, None]
    odd = ctypes.c_void_p(0x10002)
    for at, bad in ((0, None), (0, ref(NONE)), (0, ref(rows(56))), (0, ref(rows(68))), (1, None), (1, odd), (2, None), (2, odd), (3, None),
                    (3, ref(rows(56))), (4, None), (4, ref(NONE)), (4, ref(rows(ptr=0x10008))), (5, None), (5, ctypes.c_void_p(0x10010)),
                    (6, n.value - 1), (7, odd)):
        a = list(good)
        a[at] = bad
        assert L.ep_moe_few(d, *a, None) == INVALID, at
    assert L.ep_moe_few(ref(few(tokens=0)), ref(NONE), None, None, ref(NONE), ref(NONE), None, 0, None, None) == 0


def test_python_face_needs_gpu_tensors():
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    codes, scales = torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 1))
    i = torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: ep.rms_norm(x, w), lambda: ep.rms_norm_backward(x, x, w), lambda: ep.checkpoint(x),
                 lambda: ep.checkpoint_restore(codes, scales), lambda: ep.checkpoint_restore(codes, scales, dtype=torch.float32),
                 lambda: ep.moe_few_tokens(x, torch.zeros(4, 2), i, torch.zeros((2, 64, 64), dtype=torch.bfloat16),
                                           torch.zeros((2, 64, 32), dtype=torch.bfloat16)),
                 lambda: ep.rms_norm(1, w), lambda: ep.checkpoint([1])):
        with pytest.raises(ValueError):
            call()
