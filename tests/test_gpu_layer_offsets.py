"""Places past 2^31 elements: the last rows and the last experts of large tensors
have the bits of smaller ones.  (Sums are in an order that goes by the sizes, so the
smaller ones are not so small that a row has more threads.)"""
import pytest
import torch

import combine_ep_layout_06_gb300 as ep

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rand(*shape, std=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_rows_of_norm_and_checkpoints():
    rows, H = 310000, 7168                                 # 2.2e9 elements
    x = torch.zeros(rows, H, dtype=BF, device="cuda")
    x[-6:], x[1] = rand(6, H), rand(H, seed=1)
    w = rand(H, seed=2)
    small = x[-6000:].clone()
    codes, scales, total = ep.rms_norm(x, w, residual=x, quantize=True)
    for got, want in zip((codes, scales, total), ep.rms_norm(small, w, residual=small, quantize=True)):
        assert same(got[-6:], want[-6:])
    del codes, scales, total
    dx, dw = ep.rms_norm_backward(x, x, w)
    want, _ = ep.rms_norm_backward(small, small, w)
    assert same(dx[-6:], want[-6:])
    n = torch.cat([x[1:2], small[-6:]]).double()
    n = n * n / torch.sqrt((n * n).mean(-1, keepdim=True) + 1e-6)
    # all other rows are 0: the sums are those of 7 rows, rounded once (and 2^-18 as elsewhere)
    assert bool(((dw.double() - n.sum(0)).abs() <= n.sum(0).abs() * 2.0 ** -8 + n.abs().sum(0) * 2.0 ** -18).all())
    del dx
    count = torch.tensor([[2, 6]], dtype=torch.int32, device="cuda")
    offset = torch.tensor([[0, rows - 6]], dtype=torch.int32, device="cuda")
    codes, scales = ep.checkpoint(x, count, offset)
    small = small[-6:].clone()
    kept = ep.checkpoint(small)
    assert same(codes[-6:], kept[0]) and same(scales[-6:], kept[1])
    y = ep.checkpoint_restore(codes, scales, count, offset, activation="silu")
    assert same(y[-6:], ep.checkpoint_restore(*kept, activation="silu"))
    # ranks and rows far apart
    far = x.view(2, rows // 2, H)[:, -200:]
    assert same(ep.rms_norm(far, w)[1, -6:], ep.rms_norm(x[-400:].clone(), w)[-6:])
    assert same(ep.checkpoint(far)[0][1, -6:], kept[0])


def test_experts_far_into_their_weights():
    E, H, F = 96, 7168, 1792                               # up: 2.5e9 elements
    up, down = torch.zeros(E, 2 * F, H, dtype=BF, device="cuda"), torch.zeros(E, H, F, dtype=BF, device="cuda")
    for e in range(90, E):
        up[e], down[e] = rand(2 * F, H, std=H ** -0.5, seed=e), rand(H, F, std=F ** -0.5, seed=2 * e)
    x, w = rand(5, H), torch.rand(5, 4, device="cuda")
    idx = torch.tensor([[90, 91, 92, 95], [95, 94, 93, 92], [90, 95, 91, 94], [93, 92, 91, 90], [95, 95, -1, 94]], dtype=torch.int32,
                       device="cuda")
    got = ep.moe_few_tokens(x, w, idx, up, down)
    near = torch.where(idx < 0, idx, idx - 90)
    assert same(got, ep.moe_few_tokens(x, w, near, up[90:].clone(), down[90:].clone()))
    assert float(got.float().norm()) > 0 and ep.moe_error() == 0
    # little work: the other kernels
    got = ep.moe_few_tokens(x[:1, :64].contiguous(), w[:1], idx[:1], up[:, :16, :64], down[:, :64, :8])
    want = ep.moe_few_tokens(x[:1, :64].contiguous(), w[:1], near[:1], up[90:, :16, :64].clone(), down[90:, :64, :8].clone())
    assert same(got, want)
