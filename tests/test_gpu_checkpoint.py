"""Activations kept in 8 bits: saved, restored through the activation, and taken
by the expert product's gradient.

Tolerances.  The codes of bf16 rows are those of the IEEE quotient, bit for bit; of
fp16 rows the quotient may be a unit of fp32 off, so a code is within half a step
(2^-4 of the value, or 2^-10 scales) and 2^-20 more.  Restored values: finfo.eps / 2
of the result, and 2^-18 of |v| (|gate * up|) for the fp32 activation."""
import ctypes
import math

import pytest
import torch

import combine_ep_layout_06_gb300 as ep
from combine_ep_layout_06_gb300 import _lib

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
ACTS = ["none", "relu", "gelu", "silu", "swiglu"]


def rand(*shape, dtype=BF, std=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def reference(x):
    F = x.shape[-1]
    v = torch.nn.functional.pad(x.float(), (0, -F % 128)).unflatten(-1, (-1, 128))
    # fl32(a / 448): by way of 64 bits, since a tensor's division by a number multiplies by its reciprocal
    scales = (v.abs().amax(-1).double() / 448.0).float()
    codes = (v / torch.where(scales > 0, scales, 1.0)[..., None]).to(torch.float8_e4m3fn)
    codes = torch.where((scales == 0)[..., None], torch.zeros_like(codes).view(torch.uint8), codes.view(torch.uint8))
    return codes.flatten(-2)[..., :F].contiguous().view(torch.float8_e4m3fn), scales


def kept(codes, scales):
    return codes.float().double() * scales.double().repeat_interleave(128, -1)[..., :codes.shape[-1]]


def act64(v, name):
    f = torch.nn.functional
    if name == "swiglu":
        gate, up = v.chunk(2, -1)
        return f.silu(gate) * up, (gate * up).abs()
    return {"none": lambda t: t, "relu": torch.relu, "gelu": f.gelu, "silu": f.silu}[name](v), v.abs()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows,F", [(1, 8), (3, 120), (5, 128), (70, 136), (9, 328), (33, 3584), (2, 7168), (1000, 64)])
def test_save(rows, F, dtype):
    x = rand(rows, F, dtype=dtype) * torch.exp2(torch.randint(-20, 10, (rows, 1), device="cuda")).to(dtype)
    x[0, ::3] = 0.0
    x[rows // 2] = -0.0
    codes, scales = ep.checkpoint(x)
    want, want_scales = reference(x)
    assert torch.equal(scales, want_scales)
    if dtype == BF:
        assert torch.equal(codes.view(torch.uint8), want.view(torch.uint8))
    s = scales.double().repeat_interleave(128, -1)[..., :F]
    off, v = (kept(codes, scales) - x.double()).abs(), x.double().abs()
    assert bool((off <= torch.maximum(v * 2.0 ** -4, s * 2.0 ** -10) + v * 2.0 ** -20).all())


def test_blocks_that_are_not_finite():
    x = rand(4, 392)
    x[0, 5], x[1, 200], x[2, 391] = math.inf, math.nan, -math.inf
    codes, scales = ep.checkpoint(x)
    bad = torch.zeros(4, 4, dtype=torch.bool, device="cuda")
    bad[0, 0] = bad[1, 1] = bad[2, 3] = True
    assert torch.equal(scales.isnan(), bad)
    back = ep.checkpoint_restore(codes, scales)
    assert torch.equal(back.isnan(), bad.repeat_interleave(128, -1)[:, :392])
    fine = ~bad.repeat_interleave(128, -1)[:, :392]
    assert torch.equal(back[fine], kept(codes, scales)[fine].to(BF))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,N", [(1, 8), (77, 328), (40, 1792), (5, 136), (257, 64)])
def test_restore(rows, N, act, dtype):
    F = 2 * N if act == "swiglu" else N
    codes, scales = ep.checkpoint(rand(rows, F, dtype=dtype, std=2.0))
    y = ep.checkpoint_restore(codes, scales, activation=act, dtype=dtype)
    want, size = act64(kept(codes, scales), act)
    assert y.dtype == dtype and y.shape == (rows, N)
    tol = want.abs() * torch.finfo(dtype).eps / 2 + size * 2.0 ** -18 + 2.0 ** -25
    assert bool(((y.double() - want).abs() <= tol).all())
    assert torch.equal(y, ep.checkpoint_restore(codes.view(torch.uint8), scales, activation=act, dtype=dtype))


@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_groups_leave_the_other_rows(act):
    """Rows outside every group, and what the strides skip, stay as they were;
    counts past the end are cut, odd ones ignored."""
    R, rows, F = 2, 150, 272
    N = F // 2 if act == "swiglu" else F
    count, offset = ints([[70, 0, 5], [1, 100, 0]]), ints([[3, 80, 90], [0, 60, -4]])
    inside = torch.zeros(R, rows, dtype=torch.bool, device="cuda")
    for r in range(R):
        for c, o in zip(count[r].tolist(), offset[r].tolist()):
            if 0 <= o:
                inside[r, o:o + c] = True
    x = rand(R, rows, F)
    x[~inside] = math.nan
    codes = torch.full((R, rows + 1, F + 8), 77, dtype=torch.uint8, device="cuda")
    scales = torch.full((R, rows + 2, 4), 7.0, device="cuda")
    y = torch.full((R, rows, N + 16), 5.0, dtype=BF, device="cuda")
    L = _lib.load()
    desc = _lib.EpCheckpointDescC(R, 3, rows, F, 0, {"none": 0, "swiglu": 4}[act], count.data_ptr(), offset.data_ptr())

    def at(t):
        return ctypes.byref(_lib.EpRowsC(t.data_ptr(), t.stride(0), t.stride(1)))
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert L.ep_checkpoint_save(ctypes.byref(desc), at(x), at(codes), at(scales), st) == 0
    assert L.ep_checkpoint_restore(ctypes.byref(desc), at(codes), at(scales), at(y), st) == 0
    want, want_scales = reference(x)
    assert torch.equal(codes[:, :rows, :F][inside], want.view(torch.uint8)[inside])
    assert torch.equal(scales[:, :rows, :3][inside], want_scales[inside])
    assert bool((codes[:, :rows][~inside] == 77).all()) and bool((codes[:, rows:] == 77).all())
    assert bool((codes[..., F:] == 77).all()) and bool((scales[..., 3] == 7).all()) and bool((scales[:, rows:] == 7).all())
    assert bool((scales[:, :rows][~inside] == 7).all())
    assert bool((y[~inside] == 5).all()) and bool((y[..., N:] == 5).all())
    a, b = ep.checkpoint(x, count, offset)
    assert torch.equal(a.view(torch.uint8)[inside], want.view(torch.uint8)[inside]) and torch.equal(b[inside], want_scales[inside])
    z = ep.checkpoint_restore(a, b, count, offset, activation=act)
    assert torch.equal(z[inside], y[..., :N][inside])
    z = ep.checkpoint_restore(codes[:, :rows, :F], scales[:, :rows, :3], count, offset, activation=act)
    assert torch.equal(z[inside], y[..., :N][inside])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_gradient_takes_codes(act, dtype):
    """Kept values that bf16 and fp16 hold exactly (scales are powers of two):
    the gradients have the bits of those from 16-bit pre-activations."""
    R, rows, K, N = 2, 90, 128, 136
    F = 2 * N if act == "swiglu" else N
    x, w, g = rand(R, rows, K, dtype=dtype), rand(4, F, K, dtype=dtype, seed=1, std=0.1), rand(R, rows, N, dtype=dtype, seed=2)
    codes = rand(R, rows, F, seed=3, std=4.0).to(torch.float8_e4m3fn)
    scales = torch.exp2(torch.randint(-3, 2, (R, rows, -(-F // 128)), device="cuda")).float()
    pre = kept(codes, scales).to(dtype)
    assert torch.equal(pre.double(), kept(codes, scales))
    count, offset = ints([[50, 40], [0, 33]]), ints([[0, 50], [0, 7]])
    inside = torch.ones(R, rows, dtype=torch.bool, device="cuda")
    inside[1, :7], inside[1, 40:] = False, False
    want = ep.expert_product_backward(g, x, w, count, offset, pre=pre, activation=act, bias_grad=True)
    got = ep.expert_product_backward(g, x, w, count, offset, pre=codes, pre_scales=scales, activation=act, bias_grad=True)
    assert torch.equal(got[0][inside], want[0][inside])
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    got = ep.expert_product_backward(g, x, w, count, offset, pre=codes.view(torch.uint8), pre_scales=scales, activation=act)
    assert torch.equal(got[1], want[1])
    assert ep.moe_error() == 0


def test_streams_graphs_and_no_rows():
    x = rand(64, 512)
    want = ep.checkpoint(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        codes, scales = ep.checkpoint(x)
        y = ep.checkpoint_restore(codes, scales, activation="swiglu")
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = ep.checkpoint_restore(*ep.checkpoint(x, stream=side), activation="swiglu", stream=side)
    torch.cuda.synchronize()
    assert torch.equal(codes.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(y, z)
    for shape in ((0, 64), (2, 0, 64)):
        codes, scales = ep.checkpoint(torch.zeros(shape, dtype=BF, device="cuda"))
        assert codes.shape == shape and scales.shape == shape[:-1] + (1,)
        assert ep.checkpoint_restore(codes, scales, activation="swiglu").shape == shape[:-1] + (32,)


def test_refusals():
    x, n = rand(2, 6, 64), ints([[1], [2]])
    codes, scales = ep.checkpoint(x)
    w = rand(2, 64, 16)
    for call in (lambda: ep.checkpoint(x.float()), lambda: ep.checkpoint(x[0, 0]), lambda: ep.checkpoint(x[..., :12]),
                 lambda: ep.checkpoint(x[..., 4:12]), lambda: ep.checkpoint(x, n, None), lambda: ep.checkpoint(x, n.long(), n),
                 lambda: ep.checkpoint(x, ints([1, 2, 3]), ints([1, 2, 3])), lambda: ep.checkpoint(x, n, n[:1]),
                 lambda: ep.checkpoint(x.transpose(1, 2)), lambda: ep.checkpoint(x.cpu()),
                 lambda: ep.checkpoint_restore(codes, scales[..., :0]), lambda: ep.checkpoint_restore(codes, scales.double()),
                 lambda: ep.checkpoint_restore(codes.float(), scales), lambda: ep.checkpoint_restore(codes[..., :8], scales, activation="swiglu"),
                 lambda: ep.checkpoint_restore(codes, scales, activation="tanh"),
                 lambda: ep.checkpoint_restore(codes, scales, dtype=torch.float32),
                 lambda: ep.checkpoint_restore(codes[..., 4:12], scales), lambda: ep.checkpoint_restore(codes, scales[:1]),
                 lambda: ep.expert_product_backward(x, rand(2, 6, 16), w, pre=x, pre_scales=scales, activation="silu"),
                 lambda: ep.expert_product_backward(x, rand(2, 6, 16), w, pre=codes, activation="silu"),
                 lambda: ep.expert_product_backward(x, rand(2, 6, 16), w, pre_scales=scales, activation="silu")):
        with pytest.raises(ValueError):
            call()
