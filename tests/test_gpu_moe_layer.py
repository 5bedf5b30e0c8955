"""The example layer end to end (routing, dispatch, grouping, expert products,
un-grouping, combine, and back) against a dense mixture of experts in 64 bits
with autograd, given the layer's own routing.

Tolerances: the layer rounds to bf16 after every step (half a unit 2^-8); a
forward passes 4 roundings on the way (gated product, down product, weighted
un-grouping, combine), a gradient at most 8, each of sums of terms of both
signs: 2-norm errors of 4 * 2^-8 and 8 * 2^-8 of the result bound them."""
import os
import sys

import pytest
import torch

import combine_ep_layout_06_gb300 as ep

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def rel(got, want):
    return float((got.double() - want).norm() / want.norm().clamp(min=1e-30))


@pytest.mark.parametrize("W,E,k,T,H,F,ragged", [(2, 8, 2, 128, 256, 192, False), (4, 32, 4, 65, 512, 136, True),
                                                (1, 4, 1, 33, 128, 64, False)])
def test_layer_and_its_gradients(W, E, k, T, H, F, ragged):
    from moe_layer import MoeLayer
    layer = MoeLayer(W, E, k, T, H, F, seed=W)
    g = torch.Generator(device="cuda").manual_seed(7)
    layer.down_bias += (torch.randn(E, H, generator=g, device="cuda") * 0.1).to(torch.bfloat16)
    x = torch.randn(W, T, H, generator=g, device="cuda").to(torch.bfloat16)
    nt = [max(1, T - 7 * s) for s in range(W)] if ragged else [T] * W
    out, balance = layer.forward(x, num_tokens=nt)
    grad = (torch.randn(W, T, H, generator=g, device="cuda") * 0.1).to(torch.bfloat16)
    indices, logits = layer.saved[3], layer.saved[1]
    grads = layer.backward(grad, torch.full((), 3.0, device="cuda"))
    torch.cuda.synchronize()
    assert layer.op.get_error() == (0, 0) and ep.moe_error() == 0
    here = torch.arange(T, device="cuda") < torch.tensor(nt, device="cuda")[:, None]
    leaves = [t.detach().double().requires_grad_(True)
              for t in (x, layer.router, layer.gate_up, layer.down, layer.down_bias)]
    dx, router, gate_up, down, bias = leaves
    rows = dx[here]
    # the rounded logits' values, the exact ones' slopes
    exact = rows @ router.T
    lg = exact + (logits[here].double() - exact).detach()
    ids = indices[here].long()
    w = torch.softmax(lg.gather(1, ids), 1)
    v = torch.einsum("nh,efh->nef", rows, gate_up)
    hh = torch.nn.functional.silu(v[..., :F]) * v[..., F:]
    y = torch.einsum("nef,ehf->neh", hh, down) + bias
    full = (y.gather(1, ids[..., None].expand(-1, -1, H)) * w[..., None]).sum(1)
    n = rows.shape[0]
    share = torch.bincount(ids.flatten(), minlength=E).double() * E / (k * n)
    loss = (layer.balance_coef * (share * torch.softmax(lg, 1).mean(0)).sum()
            + layer.z_coef * torch.logsumexp(lg, 1).square().mean())
    assert rel(out[here], full.detach()) < 4 * 2.0 ** -8
    assert abs(float(balance) - float(loss.detach())) < 1e-5 * abs(float(loss.detach()))
    want = torch.autograd.grad((full * grad[here].double()).sum() + 3.0 * loss, leaves)
    for name, got, ref in zip(("x", "router", "gate_up", "down", "down_bias"), grads, want):
        assert rel(got, ref) < 8 * 2.0 ** -8, name


def test_example_runs(capsys):
    import moe_layer
    moe_layer.main()
    lines = capsys.readouterr().out.strip().splitlines()
    first, last = (float(s.split("error ")[1].split(",")[0]) for s in (lines[0], lines[-1]))
    assert last < first                       # it learns


@pytest.mark.parametrize("W,T,H", [(2, 64, 256), (4, 600, 512)])
def test_back_to_back_calls_are_ordered(W, T, H):
    """Kernels get ready while the one before them ends; each must still see
    all that came before it: a chain product -> route -> dispatch -> combine on
    changing inputs, with nothing waited for in between, gives the bits of the
    same chain with the GPU waited for after every call."""
    E, k, F = 4 * W, 2, 128
    g = torch.Generator(device="cuda").manual_seed(3)

    def rand(*shape):
        return (torch.randn(shape, generator=g, device="cuda") * 0.2).to(torch.bfloat16)
    w1, w2, router = rand(1, F, H), rand(1, H, F), rand(1, E, H)
    op = ep.EpDispatchCombineOp(ep.EpDispatchCombineConfig(W, E, k, H, T))

    def chain(x, wait):
        pause = torch.cuda.synchronize if wait else (lambda: None)
        h = ep.expert_product(x.view(1, W * T, H), w1, activation="silu")
        pause()
        y = ep.expert_product(h, w2, residual=x.view(1, W * T, H))
        pause()
        logits = ep.expert_product(y, router).view(W, T, E)
        pause()
        weights, idx = ep.route(logits, k)
        pause()
        op.dispatch(y.view(W, T, H), weights, None, idx)
        pause()
        op.identity_expert()
        pause()
        out, _ = op.combine()
        pause()
        dx, dw, _ = ep.expert_product_backward(out.view(1, W * T, H), h, w2)
        pause()
        return out, dx, dw
    inputs = [rand(W, T, H) for _ in range(12)]
    want = [chain(x, True) for x in inputs]
    got = [chain(x, False) for x in inputs]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert op.get_error() == (0, 0) and ep.moe_error() == 0
