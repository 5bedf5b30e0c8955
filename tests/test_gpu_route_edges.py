"""Routing and losses at the edges of their ranges: the last lane's experts,
few experts over many tokens, logits far from 0.  References and tolerances are
those of test_gpu_route."""
import pytest
import torch

import combine_ep_layout_06_gb300 as ep
from test_gpu_route import DTYPES, OPTIONS, draw_logits, near, ref_route

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
