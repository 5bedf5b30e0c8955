"""Routing and losses at the edges of their ranges: the last lane's experts,
few experts over many tokens, logits far from 0.  References and tolerances are
those of test_gpu_route."""
import pytest
import torch

import combine_ep_layout_06_gb300 as ep
from test_gpu_route import DTYPES, OPTIONS, clean, draw_logits, near, ref_loss, ref_route

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [8, 24, 40, 72, 136, 200, 264, 328, 504, 520, 600, 776, 1000, 1016, 1024])
def test_bias_up_to_the_last_expert(E):
    """Numbers of experts that end inside a lane's share (8, 16 or 32 experts a
    lane), and those that do not; the bias decides, the last expert included."""
    W, T, k = 2, 19, min(8, E)
    bias = torch.linspace(-2.0, 2.0, E)[torch.randperm(E, generator=torch.Generator().manual_seed(E))].clone()
    bias[-1] = 6.0
    for i, dtype in enumerate(DTYPES):
        x = draw_logits(W, T, E, dtype, seed=E + i)
        for score, renorm, scale in OPTIONS:
            w, idx = ep.route(x.cuda(), k, score=score, renormalize=renorm, scale=scale, bias=bias.cuda())
            rw, ridx = ref_route(x, k, score, renorm, scale, bias, [T] * W)
            assert torch.equal(idx.cpu(), ridx)
            near(w, rw, scale)


@pytest.mark.parametrize("W,T,E,k", [(8, 20000, 1, 1), (8, 20000, 2, 1), (4, 40000, 3, 2), (2, 30000, 5, 2),
                                     (2, 10000, 9, 4), (1, 1000, 513, 3)])
def test_losses_over_several_clusters(W, T, E, k):
    """Sums joined by the second kernel where some of its blocks have no
    expert, and straight to their part of the loss."""
    x = draw_logits(W, T, E, torch.float32, seed=E)
    g = torch.Generator().manual_seed(E)
    idx = torch.argsort(torch.rand((W, T, E), generator=g), -1)[..., :k].to(torch.int32).contiguous()
    nt = [T - 7 * s for s in range(W)]
    rl, rc, rp = ref_loss(clean(x), idx, nt, 0.5, 0.25)
    a = (x.cuda(), idx.cuda())
    first = ep.balance_loss(*a, balance_coef=0.5, z_coef=0.25, num_tokens=nt)
    assert torch.equal(first[1].cpu(), rc)
    near(first[0], rl, 0.0)
    near(first[2], rp, 1.0 / E)
    for _ in range(20):
        assert all(torch.equal(p, q) for p, q in zip(ep.balance_loss(*a, balance_coef=0.5, z_coef=0.25, num_tokens=nt), first))
