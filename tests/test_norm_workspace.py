"""The workspace of the norm's gradient holds a row of sums for every block, and no more than
the kernel with most blocks needs."""
import ctypes

import pytest

from combine_ep_layout_06_gb300 import _lib, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.load()


def parts(L, rows, width, dtype=0):
    d = _lib.EpNormDescC(1, rows, width, dtype, dtype, 1e-6, _lib.EpRowsC(0x10000, 0, width), 0x10000)
    n = ctypes.c_size_t(0)
    assert L.ep_rms_norm_workspace(ctypes.byref(d), ctypes.byref(n)) == 0
    assert n.value % (width * 4) == 0
    return n.value // (width * 4)


SMS = 152


@pytest.mark.parametrize("rows,width,most", [
    (1 << 20, 32768, 3 * SMS),          # a block a row: three an SM
    (1 << 20, 32767, 3 * SMS),
    (1 << 20, 16384, 3 * SMS),
    (1 << 20, 7168, 6 * SMS),           # strided threads: six blocks of 256 an SM
    (1 << 20, 256, 8 * SMS),
    (100, 7168, 100), (1, 7168, 1), (17, 33, 17)])
def test_no_more_than_the_most_blocks(L, rows, width, most):
    for dtype in (0, 2):
        assert parts(L, rows, width, dtype) <= most


def test_never_less_with_more_rows(L):
    """(A caller may size it for its largest batch.)"""
    for width in (8, 100, 264, 1024, 2048, 4096, 7168, 8192, 16384, 32768):
        for dtype in (0, 2):
            last = 0
            for rows in (1, 2, 7, 8, 100, 455, 456, 457, 912, 1215, 1216, 1217, 2431, 2432, 4863, 4864, 5000, 9727, 9728, 20000, 1 << 20):
                now = parts(L, rows, width, dtype)
                assert now >= last, (width, dtype, rows)
                last = now


@pytest.mark.gpu
@pytest.mark.parametrize("rows,width,shift", [(6000, 1024, 0), (2000, 7168, 0), (600, 32768, 0), (600, 32760, 1), (2000, 7168, 1),
                                              (20000, 264, 0), (20000, 264, 1), (300, 264, 0), (50, 4096, 1), (3000, 60, 1)])
@pytest.mark.parametrize("total", [False, True])
def test_nothing_behind_the_workspace(L, rows, width, shift, total):
    """Exactly the bytes it asks for: what follows stays, and the sums are right."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, grad, more = (torch.randn(rows * width + 8, generator=g, device="cuda").bfloat16()[shift:] for _ in range(3))
    w = torch.randn(width, generator=g, device="cuda").bfloat16()
    out, dw = torch.empty(rows * width + 8, dtype=torch.bfloat16, device="cuda")[shift:], torch.empty_like(w)

    def at(t):
        return _lib.EpRowsC(t.data_ptr(), 0, width)
    d = _lib.EpNormDescC(1, rows, width, 0, 0, 1e-6, at(x), w.data_ptr())
    n = ctypes.c_size_t(0)
    assert L.ep_rms_norm_workspace(ctypes.byref(d), ctypes.byref(n)) == 0
    scratch = torch.full((n.value + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    none = _lib.EpRowsC(None, 0, 0)
    assert L.ep_rms_norm_backward(ctypes.byref(d), ctypes.byref(at(grad)), ctypes.byref(at(more) if total else none),
                                  ctypes.byref(at(out)), dw.data_ptr(), scratch.data_ptr(), n.value, None, st) == 0
    assert bool((scratch[n.value:] == 0x5A).all())
    h = x[:rows * width].view(rows, width).double()
    u = grad[:rows * width].view(rows, width).double() * h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6)
    want, size = u.sum(0), u.abs().sum(0)
    # a rounding to bf16, and for each row an addition and 2^-18 of its term
    tol = want.abs() * 2.0 ** -8 + size * ((rows + 32) * 2.0 ** -24 + 2.0 ** -18)
    assert bool(((dw.double() - want).abs() <= tol).all())
