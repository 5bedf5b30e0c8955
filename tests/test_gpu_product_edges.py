"""Expert products at the edges: values that are not finite, tensors that
autograd follows, groups of very many rows."""
import pytest
import torch

import combine_ep_layout_06_gb300 as ep

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def test_relu_keeps_what_is_not_a_number():
    """y = max(v, 0) of a NaN is NaN, whichever lane and type; so is an infinite
    input against weights of both signs.  Other rows do not see it."""
    for dtype in (torch.bfloat16, torch.float16):
        g = torch.Generator().manual_seed(3)
        x = torch.randn((40, 64), generator=g).to(dtype)
        w = torch.randn((1, 136, 64), generator=g).to(dtype)
        x[7, 5], x[33, :2] = NAN, INF
        w[0, :, 0], w[0, :, 1] = w[0, :, 0].abs(), -w[0, :, 1].abs()        # inf - inf in row 33
        want = torch.relu(x.double() @ w[0].double().T)
        y = ep.expert_product(x.cuda(), w.cuda(), activation="relu").cpu()
        clean = [i for i in range(40) if i not in (7, 33)]
        assert torch.isnan(want[7]).all() and torch.isnan(want[33]).all()
        assert torch.isnan(y[7]).all() and torch.isnan(y[33]).all()
        u = torch.finfo(dtype).eps / 2
        # 64 products in fp32, one rounding
        tol = u * want[clean].abs() + 64 * 2.0 ** -23 * (x[clean].double().abs() @ w[0].double().abs().T) + 2.0 ** -24
        assert ((y[clean].double() - want[clean]).abs() <= tol).all()


def test_relu_gradient_of_a_closed_unit_is_zero():
    """A unit at or below 0 passes nothing on, not even an infinite gradient; an
    open one passes it on."""
    for dtype in (torch.bfloat16, torch.float16):
        g = torch.Generator().manual_seed(4)
        pre = torch.randn((24, 72), generator=g).to(dtype)
        grad = torch.randn((24, 72), generator=g).to(dtype)
        pre[5], grad[5] = -pre[5].abs() - 0.5, INF
        pre[6], grad[6] = 0.0, -INF
        pre[9, 3], grad[9, 3] = 1.0, INF
        x = torch.ones((24, 64), dtype=dtype)
        w = (torch.rand((1, 72, 64), generator=g) + 0.5).to(dtype)
        dx, dw, db = ep.expert_product_backward(grad.cuda(), x.cuda(), w.cuda(), pre=pre.cuda(), activation="relu",
                                                bias_grad=True)
        dx, dw, db = dx.cpu().double(), dw.cpu().double(), db.cpu().double()
        assert (dx[5:7] == 0).all() and (dx[9] == INF).all()
        assert (dw[0, 3] == INF).all() and db[0, 3] == INF
        d = torch.where(pre > 0, grad, torch.zeros_like(grad)).double()
        finite = [j for j in range(72) if j != 3]
        u = torch.finfo(dtype).eps / 2
        # 24 terms in fp32, one rounding
        for got, want in ((dw[0][finite], d.T[finite] @ x.double()), (db[0][finite], d.sum(0)[finite])):
            tol = u * want.abs() + 24 * 2.0 ** -23 * d[:, finite].abs().sum(0).max() + 2.0 ** -24
            assert ((got - want).abs() <= tol).all()


def test_a_group_of_very_many_rows():
    """The weight gradient of one group of almost 2^30 rows runs for more than a
    second in one pair of SMs, and no wait gives up.  Small whole numbers in a few
    rows, the first and last among them: every sum is exact."""
    n = (1 << 30) - 5
    g = torch.Generator().manual_seed(1)
    at = torch.cat([torch.tensor([0, 1, 63, 127, 128, n - 129, n - 2, n - 1]),
                    torch.randint(200, n - 200, (300,), generator=g)]).unique()
    xs, gs = (torch.randint(-2, 3, (len(at), 8), generator=g).to(torch.bfloat16) for _ in range(2))
    w = torch.randint(-2, 3, (1, 8, 8), generator=g).to(torch.bfloat16)
    x, grad = (torch.zeros((n, 8), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[at.cuda()], grad[at.cuda()] = xs.cuda(), gs.cuda()
    assert ep.moe_error() == 0
    dx, dw, db = ep.expert_product_backward(grad, x, w.cuda(), bias_grad=True)
    assert ep.moe_error() == 0
    want = gs.double() @ w[0].double()
    assert torch.equal(dx[at.cuda()].cpu().double(), want)
    assert int(torch.count_nonzero(dx)) == int(torch.count_nonzero(want))
    total = gs.double().T @ xs.double()
    assert total.abs().max() <= 256 and torch.equal(dw[0].cpu().double(), total)
    assert torch.equal(db[0].cpu().double(), gs.double().sum(0))
    y = ep.expert_product(x, w.cuda())
    want = xs.double() @ w[0].double().T
    assert torch.equal(y[at.cuda()].cpu().double(), want)
    assert int(torch.count_nonzero(y)) == int(torch.count_nonzero(want))


def test_writing_into_out_is_seen_by_autograd():
    """Another operator that saved `out` for its gradient learns that it changed."""
    x = torch.randn((16, 64)).to(torch.bfloat16).cuda()
    w = torch.randn((1, 72, 64)).to(torch.bfloat16).cuda()
    out = torch.zeros((16, 72), dtype=torch.bfloat16, device="cuda")
    p = torch.ones((16, 72), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    loss = (p * out).sum()
    before = out._version
    assert ep.expert_product(x, w, out=out) is out
    assert out._version == before + 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        other = torch.zeros_like(out)
        ep.expert_product(x, w, out=other)
    ep.expert_product(x, w, out=other)            # has no version to count
    assert torch.equal(other, out)
