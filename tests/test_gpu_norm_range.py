"""rms_norm and its gradient over fp32's whole range, against 64 bits: rows whose
squares or their sum pass fp32, and rows whose squares vanish in it.

Tolerances are those of test_gpu_norm.py: R = 2^-18 for the sums and the root, and the
output's own rounding; on top come steps of fp32's subnormals (2^-149), one for each
product that may end there."""
import pytest
import torch

import combine_ep_layout_06_gb300 as ep

pytestmark = pytest.mark.gpu

R = 2.0 ** -18
STEP = 2.0 ** -149
BF, F = torch.bfloat16, torch.float32


def rand(*shape, dtype=F, std=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def signs(*shape, seed=0):
    return rand(*shape, seed=seed).sign()


def reference(total, weight, eps):
    h = total.double()
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * weight.double()


def close(got, want, extra):
    t = torch.finfo(got.dtype)
    tol = want.abs() * (t.eps / 2 * (got.dtype != F) + R) + t.tiny * t.eps + extra
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), float((off / tol).nan_to_num(float("inf")).max())


def check_codes(codes, scales, want):
    blocks = want.unflatten(-1, (-1, 128))
    top = blocks.abs().amax(-1) / 448.0
    assert bool(((scales.double() - top).abs() <= top * R + 2 * STEP).all())
    s = scales.double()[..., None]
    off = (codes.float().double().unflatten(-1, (-1, 128)) * s - blocks).abs()
    tol = torch.maximum(blocks.abs() * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -12) + blocks.abs() * R
    assert bool((off <= tol).all()), float((off / tol).max())


def largest(rows, H, dtype):
    """Rows of the type's largest number, and of what is near the border where
    the sum of squares first passes fp32."""
    x = signs(rows, H) * float(torch.finfo(dtype).max)
    x[1::3] = rand(len(x[1::3]), H, seed=1) * 2.0 ** 57
    x[2::3] = rand(len(x[2::3]), H, seed=2).clamp(-3.9, 3.9) * 2.0 ** 126
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("H", [64, 1000, 4104, 5001, 7168, 16384, 32767, 32768])
def test_largest_values(H, dtype):
    x, w = largest(6, H, dtype), rand(H, dtype=dtype, seed=3)
    for eps in (1e-6, 2.0 ** 120):                          # nothing, and next to some squares
        close(ep.rms_norm(x, w, eps=eps), reference(x, w, eps), STEP)
        if H % 128 == 0:
            check_codes(*ep.rms_norm(x, w, eps=eps, quantize=True), reference(x, w, eps))


def root_fits(x, eps):
    """Rows whose 1 / root is an fp32 number: with eps 0 those of a root mean square of 2^-127 or more."""
    rms = x.double().square().mean(-1).sqrt()
    return rms >= 2.0 ** -127 if eps == 0 else rms >= 0


# Rows of every magnitude under every eps: from one that is all, by one that is next to the
# squares, to one that is nothing.
EPS = [0.0, 2.0 ** -149, 2.0 ** -130, 2.0 ** -101, 2.0 ** -76, 2.0 ** -75, 2.0 ** -74, 1e-6, 1.0, 2.0 ** 60, 2.0 ** 120, 2.0 ** 127]


def magnitudes(H, dtype):
    e = torch.arange(-148 if dtype == F else -132, 126, device="cuda")
    x = rand(len(e), H, seed=4).clamp(-3.9, 3.9).double() * torch.pow(2.0, e.double())[:, None]
    x[:, 0] = torch.pow(2.0, e.double())                    # no row of zeros
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("H", [1, 96, 2056, 2057])
def test_magnitudes(H, dtype):
    x, w = magnitudes(H, dtype), rand(H, dtype=dtype, seed=5)
    for eps in EPS:
        want = reference(x, w, torch.tensor(eps, dtype=F).double().item())
        ok = root_fits(x, eps)
        close(ep.rms_norm(x, w, eps=eps)[ok], want[ok], STEP * (1 + w.double().abs()))


def gradient_check(x, g, w, more, eps):
    h, v = x.double().requires_grad_(True), w.double().requires_grad_(True)
    want, want_w = torch.autograd.grad(reference(h, v, eps), (h, v), g.double())
    u = (g.double() * w.double()).abs()
    r = 1 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + eps)
    n = x.double().abs() * r
    size = R * r * (u + n * (u * n).mean(-1, keepdim=True))
    fits = root_fits(x, eps)
    x, g, more, want, size, n = (t[fits] for t in (x, g, more, want, size, n))
    want_w = (g.double() * n * x.double().sign()).sum(0)
    fits = (want.abs() + size).amax(-1) < 2.0 ** 127         # others' gradients are past fp32
    extra = size + 4 * STEP
    dx, dw = ep.rms_norm_backward(g, x, w, eps=eps)
    close(dx[fits], want[fits], extra[fits])
    rows = len(x)
    extra_w = ((rows + 32) * 2.0 ** -24 + R) * (g.double().abs() * n).sum(0) + rows * STEP
    close(dw, want_w, extra_w)
    dx, dw = ep.rms_norm_backward(g, x, w, grad_total=more, eps=eps)
    close(dx[fits], want[fits] + more[fits].double(), extra[fits] + R * more[fits].double().abs())
    close(dw, want_w, extra_w)          # in another order, where the ring has other stages
    return int(fits.sum())


# a warp a row; a block a row, few and many rows; 4 chunks a thread; the ring; strided threads
@pytest.mark.parametrize("rows,H", [(64, 256), (40, 7168), (600, 1024), (500, 16392), (480, 32768), (1300, 7168), (1300, 8192),
                                    (5000, 1024), (300, 5001), (40, 32767), (600, 77)])
@pytest.mark.parametrize("dtype", [BF, F])
def test_gradient_of_largest_values(rows, H, dtype):
    x, g, w = largest(rows, H, dtype), rand(rows, H, dtype=dtype, seed=6), rand(H, dtype=dtype, seed=7)
    more = rand(rows, H, dtype=dtype, std=2.0 ** -60, seed=8)
    assert gradient_check(x, g, w, more, 1e-6) == rows
    assert gradient_check(x, g, w, more, 2.0 ** 120) == rows
    assert ep.moe_error() == 0


@pytest.mark.parametrize("H", [1, 96, 520, 2056, 2057])
@pytest.mark.parametrize("dtype", [BF, F])
def test_gradient_of_magnitudes(H, dtype):
    x = magnitudes(H, dtype)
    g = rand(len(x), H, dtype=dtype, std=2.0 ** -30, seed=9)
    w, more = rand(H, dtype=dtype, seed=10), rand(len(x), H, dtype=dtype, std=2.0 ** -60, seed=11)
    for eps in EPS:
        if H == 1 and eps < 1e-6:
            continue                    # the gradient is a difference of equal numbers: nothing of it is left
        assert gradient_check(x, g, w, more, torch.tensor(eps, dtype=F).double().item()) > 150


def test_gradient_of_small_rows_through_the_ring():
    x, g, w = rand(5000, 1032, seed=12), rand(5000, 1032, std=2.0 ** -40, seed=13), rand(1032, seed=14)
    more = rand(5000, 1032, seed=15)
    x[::2] *= 2.0 ** -70
    x[1::4] *= 2.0 ** -100
    assert gradient_check(x, g, w, more, 0.0) == 5000
    assert ep.moe_error() == 0


@pytest.mark.parametrize("rows,H", [(1000, 1024), (2000, 2048), (600, 16392), (600, 32768), (5000, 32), (6, 256)])
@pytest.mark.parametrize("dtype", [BF, F])
def test_gradient_in_blocks_that_take_several_rows(rows, H, dtype):
    """A block a row where rows are too few for the ring, or too wide."""
    x, g, w = rand(rows, H, dtype=dtype), rand(rows, H, dtype=dtype, seed=1), rand(H, dtype=dtype, seed=2)
    assert gradient_check(x, g, w, rand(rows, H, dtype=dtype, seed=3), 1e-6) == rows
