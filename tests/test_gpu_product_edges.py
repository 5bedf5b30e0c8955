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
