"""rms_norm and its gradient against 64 bits.

Tolerances.  A row's sum of squares has only positive terms and at most 32 + 10
fp32 additions in a row, so it is within 44 * 2^-24 of its value, its reciprocal
root within half of that and two units of rsqrt: R = 2^-18 bounds every product
of it.  On top comes the output's rounding, finfo.eps / 2 of the value (or half
a step of its subnormals).  E4M3 is off by 2^-4 of the value or 2^-10 scales."""
import ctypes
import math

import pytest
import torch

import combine_ep_layout_06_gb300 as ep
from combine_ep_layout_06_gb300 import _lib

pytestmark = pytest.mark.gpu

R = 2.0 ** -18
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def rand(*shape, dtype=F, std=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def reference(total, weight, eps):
    h = total.double()
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * weight.double()


def close(got, want, extra):
    t = torch.finfo(got.dtype)
    tol = want.abs() * (t.eps / 2 * (got.dtype != F) + R) + t.tiny * t.eps + extra
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), float((off / tol).max())


def check_codes(codes, scales, want):
    blocks = want.unflatten(-1, (-1, 128))
    top = blocks.abs().amax(-1) / 448.0
    assert bool(((scales.double() - top).abs() <= top * R + 2.0 ** -149).all())
    s = scales.double()[..., None]
    off = (codes.float().double().unflatten(-1, (-1, 128)) * s - blocks).abs()
    tol = torch.maximum(blocks.abs() * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -12) + blocks.abs() * R
    assert bool((off <= tol).all()), float((off / tol).max())


@pytest.mark.parametrize("dtype", [BF, HF, F])
@pytest.mark.parametrize("rows,H", [(1, 1), (3, 7), (5, 8), (1, 7168), (9, 256), (64, 129), (2, 1000), (33, 1024),
                                    (17, 2048), (4, 4104), (7, 8192), (300, 5001), (2, 16384), (3, 32768)])
def test_norm_and_total(rows, H, dtype):
    x, res, w = rand(rows, H, dtype=dtype), rand(rows, H, dtype=dtype, std=3.0, seed=1), rand(H, dtype=dtype, seed=2)
    y = ep.rms_norm(x, w)
    assert y.dtype == dtype
    close(y, reference(x, w, 1e-6), 0.0)
    y, total = ep.rms_norm(x, w, residual=res, eps=1e-3)
    assert torch.equal(total, (x.float() + res.float()).to(dtype))
    close(y, reference(total, w, 1e-3), 0.0)
    w32 = rand(H, seed=3)
    close(ep.rms_norm(x, w32), reference(x, w32, 1e-6), 0.0)


@pytest.mark.parametrize("dtype", [BF, HF, F])
@pytest.mark.parametrize("rows,H", [(1, 128), (37, 256), (3, 7168), (21, 1152), (2, 32768)])
def test_codes(rows, H, dtype):
    x, res, w = rand(rows, H, dtype=dtype), rand(rows, H, dtype=dtype, seed=1), rand(H, dtype=dtype, seed=2)
    codes, scales = ep.rms_norm(x, w, quantize=True)
    assert codes.dtype == torch.float8_e4m3fn and scales.shape == (rows, H // 128)
    check_codes(codes, scales, reference(x, w, 1e-6))
    codes, scales, total = ep.rms_norm(x, w, residual=res, quantize=True)
    assert torch.equal(total, (x.float() + res.float()).to(dtype))
    check_codes(codes, scales, reference(total, w, 1e-6))


def test_layouts():
    """Ranks, strided rows, addresses that 16-byte accesses do not reach, more
    dimensions, no rows: the bits are those of dense rows."""
    x, w = rand(6, 264, dtype=BF), rand(256, dtype=BF, seed=1)
    for off in (0, 1, 8):
        part = x[:, off:off + 256]
        want, wc = ep.rms_norm(part.contiguous(), w), ep.rms_norm(part.contiguous(), w, quantize=True)
        assert torch.equal(ep.rms_norm(part, w), want)
        a, b = ep.rms_norm(part, w, quantize=True)
        assert torch.equal(a.view(torch.uint8), wc[0].view(torch.uint8)) and torch.equal(b, wc[1])
        ranks = x.view(2, 3, 264)[:, :2, off:off + 256]
        assert torch.equal(ep.rms_norm(ranks, w), want.view(2, 3, 256)[:, :2])
        y, total = ep.rms_norm(ranks, w, residual=ranks)
        assert torch.equal(total, ranks * 2)
    deep = rand(2, 3, 4, 64, dtype=HF)
    w = rand(64, dtype=HF)
    assert torch.equal(ep.rms_norm(deep, w).view(24, 64), ep.rms_norm(deep.view(24, 64), w))
    assert torch.equal(ep.rms_norm(deep[0, 0, 0], w), ep.rms_norm(deep.view(24, 64), w)[0])
    shifted = rand(65, dtype=HF)[1:]
    close(ep.rms_norm(deep, shifted), reference(deep, shifted, 1e-6), 0.0)
    for shape in ((0, 64), (2, 0, 64), (0, 3, 64)):
        e = torch.zeros(shape, dtype=HF, device="cuda")
        assert ep.rms_norm(e, w).shape == shape
        dx, dw = ep.rms_norm_backward(e, e, w)
        assert dx.shape == shape and bool((dw == 0).all())


def test_values_at_the_edges():
    inf, nan = math.inf, math.nan
    x = rand(8, 256, dtype=BF)
    x[1] = 0
    x[2, 3] = inf
    x[3, 5] = nan
    x[4] *= 2.0 ** 120                      # squares past fp32
    x[5] *= 2.0 ** -120
    x[6] = torch.finfo(BF).max
    w = rand(256, dtype=BF, seed=1).abs() + 0.5
    y = ep.rms_norm(x, w)
    ok = torch.tensor([0, 1, 4, 5, 6, 7], device="cuda")
    close(y[ok], reference(x[ok], w, 1e-6), 0.0)
    assert bool(y[3].isnan().all())
    assert bool(y[2, 3].isnan()) and bool((y[2, :3] == 0).all())
    assert bool(ep.rms_norm(x[1:2], w, eps=0.0).isnan().all())      # 0 / 0
    codes, scales = ep.rms_norm(x, w, quantize=True)
    check_codes(codes[ok], scales[ok], reference(x[ok], w, 1e-6))
    assert bool((scales[1] == 0).all()) and bool((codes[1].view(torch.uint8) == 0).all())
    assert bool(scales[3].isnan().all()) and bool(codes[3].float().isnan().all())
    assert bool(scales[2, 0].isnan()) and bool((scales[2, 1] == 0).item())
    g = rand(8, 256, dtype=BF, seed=2)
    dx, _ = ep.rms_norm_backward(g, x, w)
    h = x[ok].double().requires_grad_(True)
    want, = torch.autograd.grad(reference(h, w, 1e-6), h, g[ok].double())
    u = (g[ok].double() * w.double()).abs()
    r = 1 / torch.sqrt(x[ok].double().square().mean(-1, keepdim=True) + 1e-6)
    n = x[ok].double().abs() * r
    close(dx[ok], want, R * r * (u + n * (u * n).mean(-1, keepdim=True)) + 2.0 ** -133)
    assert bool(dx[3].isnan().all())


@pytest.mark.parametrize("dtype,wtype", [(BF, BF), (HF, F), (F, F)])
@pytest.mark.parametrize("rows,H", [(1, 1), (4, 9), (1, 7168), (700, 264), (333, 1001), (50, 2056), (1300, 512), (310, 4096),
                                    (20, 20000), (3, 32768)])
def test_gradient(rows, H, dtype, wtype):
    x, g, w = rand(rows, H, dtype=dtype), rand(rows, H, dtype=dtype, seed=1), rand(H, dtype=wtype, seed=2)
    more = rand(rows, H, dtype=dtype, seed=3)
    h, v = x.double().requires_grad_(True), w.double().requires_grad_(True)
    want, want_w = torch.autograd.grad(reference(h, v, 1e-6), (h, v), g.double())
    u = (g.double() * w.double()).abs()
    r = 1 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + 1e-6)
    n = x.double().abs() * r
    size = R * r * (u + n * (u * n).mean(-1, keepdim=True))
    dx, dw = ep.rms_norm_backward(g, x, w)
    assert dx.dtype == dtype and dw.dtype == wtype
    close(dx, want, size)
    # one addition for a row, and R for the normed value
    close(dw, want_w, ((rows + 32) * 2.0 ** -24 + R) * (g.double().abs() * n).sum(0))
    dx, again = ep.rms_norm_backward(g, x, w, grad_total=more)
    close(dx, want + more.double(), size + R * more.double().abs())
    assert torch.equal(dw, again)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("rows,H", [(5000, 1032), (2500, 4096), (2000, 8192), (20000, 264), (3000, 77), (2000, 1537)])
def test_gradient_of_many_rows(rows, H, dtype):
    """Rows that come through shared memory ahead of their use, and rows strided by
    threads; some whose squares do not fit fp32, some with NaN."""
    x, g, w = rand(rows, H, dtype=dtype), rand(rows, H, dtype=dtype, seed=1), rand(H, dtype=dtype, seed=2)
    more = rand(rows, H, dtype=dtype, seed=3)
    x[7::100] *= 2.0 ** 100
    x[rows - 1] = math.nan
    ok = torch.arange(rows, device="cuda") != rows - 1
    h = x[ok].double().requires_grad_(True)
    want, = torch.autograd.grad(reference(h, w, 1e-6), h, g[ok].double())
    u = (g[ok].double() * w.double()).abs()
    r = 1 / torch.sqrt(x[ok].double().square().mean(-1, keepdim=True) + 1e-6)
    n = x[ok].double().abs() * r
    size = R * r * (u + n * (u * n).mean(-1, keepdim=True))
    dx, dw = ep.rms_norm_backward(g, x, w)
    close(dx[ok], want, size + 2.0 ** -133)
    assert bool(dx[rows - 1].isnan().all()) and bool(dw.isnan().all())
    dx, _ = ep.rms_norm_backward(g, x, w, grad_total=more)
    close(dx[ok], want + more[ok].double(), size + R * more[ok].double().abs())
    x[rows - 1] = 1.0
    n = x.double() / torch.sqrt(x.double().square().mean(-1, keepdim=True) + 1e-6)
    _, dw = ep.rms_norm_backward(g, x, w)
    close(dw, (g.double() * n).sum(0), ((rows + 32) * 2.0 ** -24 + R) * (g.double() * n).abs().sum(0))
    assert ep.moe_error() == 0


@pytest.mark.parametrize("rows,H", [(6, 256), (3000, 1024), (5, 77), (2000, 300)])
def test_in_place(rows, H):
    """total over x or over the residual, grad_x over grad_total: the bits of separate ones."""
    x, res, g, w = rand(rows, H, dtype=BF), rand(rows, H, dtype=BF, seed=1), rand(rows, H, dtype=BF, seed=2), rand(H, dtype=BF, seed=3)
    L, ref, none = _lib.load(), ctypes.byref, _lib.EpRowsC(None, 0, 0)
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def at(t):
        return _lib.EpRowsC(t.data_ptr(), 0, H)

    def desc(t):
        return _lib.EpNormDescC(1, rows, H, 0, 0, 1e-6, at(t), w.data_ptr())
    want, total = ep.rms_norm(x, w, residual=res)
    for over in (0, 1):
        a, b, y = x.clone(), res.clone(), torch.empty_like(x)
        assert L.ep_rms_norm(ref(desc(a)), ref(at(b)), ref(at((a, b)[over])), ref(at(y)), ref(none), st) == 0
        assert torch.equal(y, want) and torch.equal((a, b)[over], total)
    want, dw = ep.rms_norm_backward(g, total, w, grad_total=res)
    n = ctypes.c_size_t(0)
    assert L.ep_rms_norm_workspace(ref(desc(total)), ref(n)) == 0
    scratch, got_w, both = torch.empty(n.value, dtype=torch.uint8, device="cuda"), torch.empty_like(w), res.clone()
    assert L.ep_rms_norm_backward(ref(desc(total)), ref(at(g)), ref(at(both)), ref(at(both)), got_w.data_ptr(), scratch.data_ptr(),
                                  n.value, None, st) == 0
    assert torch.equal(both, want) and torch.equal(got_w, dw)


def test_gradient_against_differences():
    x, g, w = rand(11, 200), rand(11, 200, seed=1), rand(200, seed=2)
    dx, dw = ep.rms_norm_backward(g, x, w, eps=1e-2)
    for seed in range(4):
        vx, vw = rand(11, 200, seed=10 + seed).double(), rand(200, seed=20 + seed).double()
        step = 1e-5
        ends = [(reference(x.double() + s * vx, w.double() + s * vw, 1e-2) * g.double()).sum() for s in (step, -step)]
        slope = float(ends[0] - ends[1]) / (2 * step)
        mine = float((dx.double() * vx).sum() + (dw.double() * vw).sum())
        size = float((dx.double() * vx).abs().sum() + (dw.double() * vw).abs().sum())
        assert abs(slope - mine) <= size * 2.0 ** -16        # R and the differences' own 1e-10


def test_gradient_layouts():
    x, g, more = (rand(2, 5, 300, dtype=BF, seed=s) for s in range(3))
    w = rand(256, dtype=BF, seed=4)
    for off in (0, 4, 8):
        parts = [t[:, 1:4, off:off + 256] for t in (x, g, more)]
        dense = [t.contiguous() for t in parts]
        a, b = ep.rms_norm_backward(parts[1], parts[0], w, grad_total=parts[2])
        c, d = ep.rms_norm_backward(dense[1], dense[0], w, grad_total=dense[2])
        assert torch.equal(a, c) and torch.equal(b, d)


def test_streams_and_graphs():
    x, res, w = rand(64, 1024, dtype=BF), rand(64, 1024, dtype=BF, seed=1), rand(1024, dtype=BF, seed=2)
    want, grads = ep.rms_norm(x, w, residual=res, quantize=True), ep.rms_norm_backward(res, x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ep.rms_norm(x, w, residual=res, quantize=True, stream=side)
    both = ep.rms_norm_backward(res, x, w, stream=side)
    side.synchronize()
    for a, b in zip(got + both, want + grads):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ep.rms_norm(x, w, residual=res, quantize=True)
        both = ep.rms_norm_backward(res, x, w)
    x.copy_(rand(64, 1024, dtype=BF, seed=9))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got + both, ep.rms_norm(x, w, residual=res, quantize=True) + ep.rms_norm_backward(res, x, w)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_refusals():
    x, w = rand(4, 64, dtype=BF), rand(64, dtype=BF)
    for call in (lambda: ep.rms_norm(x.double(), w), lambda: ep.rms_norm(x.to(torch.int32), w), lambda: ep.rms_norm(x, w[:32]),
                 lambda: ep.rms_norm(x, w.half()), lambda: ep.rms_norm(x, w.cpu()), lambda: ep.rms_norm(x, w.view(1, 64)),
                 lambda: ep.rms_norm(x.t(), rand(4, dtype=BF)), lambda: ep.rms_norm(x[:1].expand(4, 64), w),
                 lambda: ep.rms_norm(x, w, residual=x[:2]), lambda: ep.rms_norm(x, w, residual=x.half()),
                 lambda: ep.rms_norm(x, w, eps=-1.0), lambda: ep.rms_norm(x, w, eps=math.nan),
                 lambda: ep.rms_norm(x, w, quantize=True), lambda: ep.rms_norm(x.view(2, 2, 64).transpose(0, 1), w, residual=1),
                 lambda: ep.rms_norm(rand(1, 32769), rand(32769)), lambda: ep.rms_norm(x[:, :0], w[:0]),
                 lambda: ep.rms_norm_backward(x[:2], x, w), lambda: ep.rms_norm_backward(x, x, w, grad_total=x.half()),
                 lambda: ep.rms_norm_backward(x.float(), x, w),
                 lambda: ep.rms_norm(rand(2, 2, 2, 64).transpose(0, 1), rand(64))):
        with pytest.raises(ValueError):
            call()
