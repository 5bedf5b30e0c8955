"""moe_few_tokens on each of its two ways, the kernels for little work and those on
tensor cores: every case says which one it is meant for, by the rule that the library
chooses by, so that another rule fails here and does not move cases from one to the other.

Tolerance.  test_gpu_few_tokens.py's, or where a test says so: fp32 sums of K terms are
within K * 2^-24 of the sum of magnitudes, and activations between the products within
2^-16 of their value, in fp16 on tensor cores at least within 2^-32."""
import math
import os
import re

import pytest
import torch

import combine_ep_layout_06_gb300 as ep
from test_gpu_few_tokens import call, check, make, reference

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
SOURCE = os.path.join(os.path.dirname(ep.__file__), "csrc", "ep_few.cu")
SMALL, SHIFT = map(int, re.search(r"kSmallBytes = (\d+) << (\d+);", open(SOURCE).read()).groups())
SMALL <<= SHIFT


def on(way, c):
    """c, whose weights over all choices are few bytes ("little") or not ("tensor")."""
    choices = c["indices"].numel()
    E, wide, H = c["up"].shape
    size = choices * H * (wide + c["down"].shape[2]) * 2
    assert (size > SMALL) == (way == "tensor"), (size, SMALL)
    return c


SIZES = {"little": (5, 4, 2, 256, 192), "tensor": (12, 6, 3, 1032, 776)}       # T, E, k, H, F


def one_hot_layer(way, values, x):
    """A layer in fp16 whose activations between the products are known without a
    sum: products of x and fp16 numbers near values / x, in some order for every expert."""
    T, E, k, H, F = SIZES[way]
    c = on(way, make(T, E, k, H, F, act="none", dtype=HF))
    g = torch.Generator(device="cuda").manual_seed(7)
    c["x"].zero_()
    c["x"][:, 3] = x
    pick = torch.randint(len(values), (E, F), generator=g, device="cuda")
    sign = torch.randint(0, 2, (E, F), generator=g, device="cuda") * 2 - 1
    c["up"].zero_()
    c["up"][:, :, 3] = (values.to("cuda")[pick] / x * sign).to(HF)
    return c


def one_hot_check(c, way):
    h = c["up"][:, :, 3].double() * c["x"][0, 3].double()  # [E][F], exact in fp32
    want = torch.zeros(c["x"].shape, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(want)
    F = h.shape[1]
    for t, ids in enumerate(c["indices"].tolist()):
        for j, e in enumerate(ids):
            w, down = float(c["weights"][t, j]), c["down"][e].double()
            want[t] += w * (down @ h[e])
            off = h[e].abs() * 2.0 ** -16
            if way == "tensor":
                off = off.clamp_min(2.0 ** -32)
            tol[t] += abs(w) * (down.abs() @ (off + h[e].abs() * (F + 64) * 2.0 ** -24))
    got = call(c)
    off = (got.double() - want).abs()
    tol += want.abs() * torch.finfo(HF).eps / 2 + 2.0 ** -25
    assert bool((off <= tol).all()), float((off / tol).nan_to_num(math.inf).max())
    return got


@pytest.mark.parametrize("way", ["little", "tensor"])
@pytest.mark.parametrize("at", [2.0 ** -21, 2.0 ** -17, 2.0 ** -13, 2.0 ** -6])
def test_small_activations_of_fp16(way, at):
    c = one_hot_layer(way, at * torch.linspace(0.5, 1.0, 37), max(at, 2.0 ** -14) * 1.37)
    c["down"] *= min(2.0 ** -6 / at, 4096.0)                # outputs far from fp16's smallest
    one_hot_check(c, way)


@pytest.mark.parametrize("way", ["little", "tensor"])
@pytest.mark.parametrize("most", [60000.0, 131008.0, 1040000.0])
def test_large_activations_of_fp16(way, most):
    c = one_hot_layer(way, most * torch.linspace(0.3, 1.0, 37), 23.0)
    c["down"] *= 2.0 ** -7
    assert bool(one_hot_check(c, way).isfinite().all())


def test_where_activations_of_fp16_become_infinite():
    """Up to 2^20 on tensor cores; the kernels for little work keep fp32."""
    for way in ("little", "tensor"):
        c = one_hot_layer(way, torch.tensor([2.0 ** 20]), 256.0)
        c["down"] = (c["down"].abs() + 2.0 ** -6) * 2.0 ** -10
        c["up"].abs_()
        got = call(c)
        assert bool((got.isinf() if way == "tensor" else got.isfinite()).all())
        c["x"][:, 3] = 255.0
        assert bool(call(c).isfinite().all())
    assert ep.moe_error() == 0


@pytest.mark.parametrize("way", ["little", "tensor"])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_infinite_weights(way, dtype):
    """An infinite weight of down makes its outputs infinite, by the activation's sign,
    in 64 bits as in both ways; the others stay."""
    T, E, k, H, F = SIZES[way]
    c = on(way, make(T, E, k, H, F, act="gelu", dtype=dtype))
    clean = call(c)
    c["down"][1, 5, 7], c["down"][2, 6, 8] = math.inf, -math.inf
    c["down"][3 % E, 9, 1], c["down"][3 % E, 9, 2] = math.inf, math.nan
    got, (want, _) = call(c), reference(c)
    assert torch.equal(got.isnan(), want.isnan()) and bool(want.isnan().any())
    assert torch.equal(got.isinf(), want.isinf()) and int(want.isinf().sum()) > 2
    assert torch.equal(got[want.isinf()].sign().double(), want[want.isinf()].sign())
    assert torch.equal(got[want.isfinite()], clean[want.isfinite()])


def padded(t, pad):
    """t's values as a slice of a tensor with longer rows, NaN around them."""
    big = torch.full(t.shape[:-1] + (t.shape[-1] + pad,), math.nan, dtype=t.dtype, device="cuda")
    big[..., :t.shape[-1]] = t
    return big[..., :t.shape[-1]]


@pytest.mark.parametrize("way", ["little", "tensor"])
@pytest.mark.parametrize("act,dtype", [("swiglu", BF), ("gelu", HF)])
def test_layouts_of_both_ways(way, act, dtype):
    """Ranks of tokens, strided rows, ranks of strided rows, and experts' slices of
    larger tensors have the bits of dense ones."""
    T, E, k, H, F = (6, 5, 2, 256, 64) if way == "little" else (12, 5, 4, 1032, 776)
    c = on(way, make(T, E, k, H, F, act=act, dtype=dtype, bias=True, residual=True))
    want = call(c)
    check(want, c)
    ranks = {n: c[n].view(3, T // 3, -1) for n in ("x", "residual", "weights", "indices")}
    assert torch.equal(call(dict(c, **ranks)).view(T, H), want)
    single = {n: c[n].view(T, 1, -1) for n in ("x", "residual", "weights", "indices")}
    assert torch.equal(call(dict(c, **single)).view(T, H), want)
    pads = dict(x=16, residual=8, up=24, down=8)
    for names in [[n] for n in pads] + [list(pads)]:
        assert torch.equal(call(dict(c, **{n: padded(c[n], pads[n]) for n in names})), want), names
    for n in ("x", "residual"):                            # ranks whose rows are padded
        ranks[n] = padded(c[n], pads[n]).view(3, T // 3, H)
    assert torch.equal(call(dict(c, **ranks)).view(T, H), want)
    wide = c["up"].shape[1]
    more = dict(up=torch.cat([c["up"], torch.full_like(c["up"], math.nan)], 1)[:, :wide],
                down=torch.cat([c["down"], torch.full_like(c["down"], math.nan)], 1)[:, :H])
    assert torch.equal(call(dict(c, **more)), want)


# As in test_gpu_few_tokens.py, but on tensor cores: fewest features and deepest inner size, narrow
# layers of many experts, tiles of 3 and 9 features, small depths of both products.
@pytest.mark.parametrize("T,E,k,H,F", [(64, 40, 32, 8, 968), (64, 300, 32, 264, 72), (48, 300, 30, 264, 96), (8, 6, 3, 1032, 776),
                                       (20, 5, 4, 2056, 136), (63, 40, 30, 136, 264)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_formula_on_tensor_cores(T, E, k, H, F, dtype):
    c = on("tensor", make(T, E, k, H, F, dtype=dtype, bias=T % 2 == 0, residual=T % 3 == 0, seed=T))
    if H > 1024:                                           # more terms than the bound is for: the whole
        got, (want, _) = call(c), reference(c)
        assert float((got.double() - want).norm()) <= float(want.norm()) * (torch.finfo(dtype).eps / 2 + 2.0 ** -13)
    else:
        check(call(c), c)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu", "swiglu"])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_activations_on_tensor_cores(act, dtype):
    c = on("tensor", make(16, 6, 3, 1000, 776, act=act, dtype=dtype, bias=True, residual=True, seed=5))
    check(call(c), c)


@pytest.mark.parametrize("T,E,k,H,F", [(9, 43, 3, 4000, 96), (17, 7, 1, 4168, 136)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_few_tiles_of_a_deep_product_on_tensor_cores(T, E, k, H, F, dtype):
    c = on("tensor", make(T, E, k, H, F, dtype=dtype, bias=T % 2 == 0, residual=True, seed=T))
    c["indices"][0] = -1
    got, (want, _) = call(c), reference(c)
    assert float((got.double() - want).norm()) <= float(want.norm()) * (torch.finfo(dtype).eps / 2 + 2.0 ** -13)
    for _ in range(20):
        assert torch.equal(call(c), got)
    assert ep.moe_error() == 0
