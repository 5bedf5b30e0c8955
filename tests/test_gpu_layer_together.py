"""Norm, checkpoints and the experts of a few tokens as a layer uses them: with
routing, dispatch, grouping and the expert products of the same package.

Tolerances: a step that rounds to bf16 is off by finfo.eps / 2 = 2^-8 of its value
at most; 2-norm errors of n such steps are bounded by n * 2^-8.  E4M3 codes are off
by 2^-4 of the value at most."""
import os
import sys

import pytest
import torch

import combine_ep_layout_06_gb300 as ep

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rand(*shape, std=1.0, seed=0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def rel(got, want):
    return float((got.double() - want.double()).norm() / want.double().norm().clamp(min=1e-30))


@pytest.mark.parametrize("W,T,E,k,H,F", [(2, 9, 8, 2, 256, 192), (1, 1, 16, 4, 512, 136), (4, 16, 32, 8, 128, 64),
                                         (1, 64, 4, 2, 1024, 1024)])
def test_few_tokens_agree_with_dispatch(W, T, E, k, H, F):
    """The same tokens, once through moe_few_tokens and once through dispatch,
    grouping, two products, un-grouping and combine (4 roundings there, 1 here)."""
    from moe_layer import MoeLayer
    layer = MoeLayer(W, E, k, T, H, F, seed=3)
    layer.down_bias += rand(E, H, std=0.1)
    x = rand(W, T, H, seed=1)
    present = [max(1, T - s) for s in range(W)]
    out, _ = layer.forward(x, num_tokens=present)
    logits = torch.matmul(x, layer.router.T)
    weights, indices = ep.route(logits, k, num_tokens=present)
    few = ep.moe_few_tokens(x, weights, indices, layer.gate_up, layer.down, down_bias=layer.down_bias)
    here = torch.arange(T, device="cuda") < torch.tensor(present, device="cuda")[:, None]
    assert rel(few[here], out[here]) < 5 * 2.0 ** -8
    assert bool((few[~here] == 0).all())
    assert layer.op.get_error() == (0, 0) and ep.moe_error() == 0


def test_decode_through_layers_in_a_graph():
    """A few decode steps through three layers, captured: bit for bit the eager ones."""
    from moe_layer import MoeLayer
    layers = [MoeLayer(1, 8, 2, 4, 256, 192, seed=s) for s in range(3)]
    x, residual = rand(4, 256, seed=5), rand(4, 256, seed=6)

    def step(x, total):
        for layer in layers:
            x, total = layer.decode(x, total)
        return ep.rms_norm(x, layers[0].norm, residual=total)
    want = step(x, residual)
    # against 64 bits, with the layer's own routing
    d, total = x.double(), residual.double()
    for layer in layers:
        total = total + d
        y = total / torch.sqrt((total * total).mean(-1, keepdim=True) + 1e-6)
        d = torch.zeros_like(total)
        w, ids = ep.route(torch.matmul(y.to(BF), layer.router.T), 2)
        for t in range(4):
            for j in range(2):
                e = int(ids[t, j])
                v = layer.gate_up[e].double() @ y[t]
                h = torch.nn.functional.silu(v[:192]) * v[192:]
                d[t] += float(w[t, j]) * (layer.down[e].double() @ h)
    # three layers of norm, router logits, experts and two sums each
    assert rel(want[1], total + d) < 3 * 5 * 2.0 ** -8
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x, residual)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert ep.moe_error() == 0


@pytest.mark.parametrize("W,E,k,T,H,F", [(2, 8, 2, 128, 256, 192), (4, 32, 4, 65, 512, 136)])
def test_checkpoints_in_training(W, E, k, T, H, F):
    """Training with 8-bit checkpoints: the forward pass keeps its bits, the
    gradients are those of pre-activations that are off by 2^-4 at most.  By a
    change of 2^-4 of its argument the activation's slope, and so each term of a
    gradient, changes by less than 2^-3: 2-norms by less than 2^-3, and by more than
    nothing, or the checkpoints were not what the gradient read."""
    from moe_layer import MoeLayer
    plain, kept = (MoeLayer(W, E, k, T, H, F, seed=W, checkpoints=c) for c in (False, True))
    x, g = rand(W, T, H, seed=7), rand(W, T, H, std=0.1, seed=8)
    one = torch.ones((), device="cuda")
    a, b = plain.forward(x), kept.forward(x)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert kept.saved[7] is None and kept.saved[8][0].element_size() == 1
    want, got = plain.backward(g, one), kept.backward(g, one)
    for name, p, q in zip(("x", "router", "gate_up", "down", "down_bias"), want, got):
        assert rel(q, p) < 2.0 ** -3, name
    assert rel(got[2], want[2]) > 2.0 ** -9 and torch.equal(got[4], want[4])
    assert kept.op.get_error() == (0, 0) and ep.moe_error() == 0


def test_norm_in_8_bits_through_dispatch():
    """Codes and scales of the norm go out as a pre-quantised dispatch, its
    grouped rows come back as rows of a product."""
    W, T, E, k, H, F = 2, 40, 8, 2, 256, 128
    x, residual, weight = rand(W, T, H), rand(W, T, H, seed=1), rand(H, seed=2)
    codes, scales, total = ep.rms_norm(x, weight, residual=residual, quantize=True)
    weights, indices = ep.route(rand(W, T, E, seed=3), k)
    op = ep.EpDispatchCombineOp(ep.EpDispatchCombineConfig(W, E, k, H, T, dispatch_dtype="fp8_e4m3",
                                                           max_grouped_rows_per_rank=W * T * k))
    op.dispatch(codes, weights, scales, indices)
    rows8, scales8, count, offset = op.moe_group()
    rows = ep.checkpoint_restore(rows8, scales8, count, offset)
    up = rand(E, F, H, std=H ** -0.5, seed=4)
    got = ep.expert_product(rows, up, count, offset)
    values = (codes.float() * scales.repeat_interleave(128, -1)).view(W * T, H)
    src, entry = op.src_pos.long(), op.moe_src.long()
    for r in range(W):
        for e in range(E // W):
            at = slice(int(offset[r, e]), int(offset[r, e]) + int(count[r, e]))
            token = src[r][entry[r, at] // k]
            assert torch.equal(rows[r, at], values[token].to(BF))
            if token.numel():
                assert rel(got[r, at], values[token].double() @ up[r * (E // W) + e].double().T) < 2 * 2.0 ** -8
    y, again = ep.rms_norm(x, weight, residual=residual)
    assert torch.equal(again, total)
    assert rel(values.view(W, T, H), y) < 2.0 ** -4
    assert op.get_error() == (0, 0) and ep.moe_error() == 0
