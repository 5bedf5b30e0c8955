"""Routing and losses at the edges of their ranges: the last lane's experts,
few experts over many tokens, logits far from 0.  References and tolerances are
those of test_gpu_route; a NaN is never near anything here."""
import math

import pytest
import torch

import combine_ep_layout_06_gb300 as ep
from test_gpu_route import (DTYPES, OPTIONS, TINY, UNIT, clean, draw_logits, ref_loss, ref_route, softmax,
                            weights_of)

pytestmark = pytest.mark.gpu


def near(got, want, scale, dtype=torch.float32):
    """Within 1e-5 of the largest term `scale` (one, or one per row) and of the
    result, and half a unit of a 16-bit type's last place."""
    got, want = got.cpu().double(), want.detach()
    tol = 1e-5 * scale + (UNIT[dtype] + 1e-5) * want.abs() + TINY[dtype]
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])


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


LARGE = [6e4, 1e5, 1e9, 1e10, 1e20, 9e29, 3e38]


def large_rows(E, dtype, most=3.4e38):
    """Rows whose largest logit is far from 0, of both signs: all equal, next
    to closed experts, alone, one of two, and with neighbours a few units away."""
    rows = []
    for v in LARGE:
        v = min(v, float(torch.finfo(dtype).max))
        if v > most:
            continue
        for s in (v, -v):
            rest = -v if s < 0 else 0.0
            rows += [[s] * E, [s, -math.inf] * (E // 2) + [s] * (E % 2), [s] + [rest * 2 if s < 0 else rest] * (E - 1),
                     [rest * 2 if s < 0 else rest] * (E - 2) + [s, s], [s - 0.75 * (j % 7) for j in range(E)]]
    x = torch.tensor(rows, dtype=torch.float64)
    return x.clamp(min=-float(torch.finfo(dtype).max)).where(x > -math.inf, x).to(dtype)[None]


def largest(want, terms):
    """A row's largest term: `terms`, or its largest output."""
    return want.abs().amax(-1, keepdim=True).clamp(min=terms)


@pytest.mark.parametrize("E", [12, 256, 600])
@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_far_from_zero(E, dtype):
    """Finite logits of any size (a mask's fill value over a whole row, a router
    that ran away) have finite probabilities, weights and gradients."""
    x, k = large_rows(E, dtype), 3
    nt = [x.shape[1]]
    g = torch.Generator().manual_seed(E)
    gw = torch.randn((1, nt[0], k), generator=g)
    cb, cz = 0.5, 0.25
    for score, renorm, scale in OPTIONS:
        w, idx = ep.route(x.cuda(), k, score=score, renormalize=renorm, scale=scale)
        rw, ridx = ref_route(x, k, score, renorm, scale, None, nt)
        assert torch.equal(idx.cpu(), ridx) and torch.isfinite(w).all()
        near(w, rw, scale)
        xs = clean(x).requires_grad_(True)
        want, = torch.autograd.grad((weights_of(xs, ridx.long(), score, renorm, scale) * gw).sum(), xs)
        got = ep.route_backward(gw.cuda(), x.cuda(), idx, score=score, renormalize=renorm, scale=scale)
        want = torch.nan_to_num(want, nan=0.0)
        near(got, want, largest(want, 4 * scale * float(gw.abs().max())), dtype)
    idx = torch.argsort(torch.rand((1, nt[0], E), generator=g), -1)[..., :k].to(torch.int32).contiguous()
    rl, rc, rp = ref_loss(clean(x), idx, nt, cb, cz)
    loss, counts, probs = ep.balance_loss(x.cuda(), idx.cuda(), balance_coef=cb, z_coef=cz)
    assert torch.equal(counts.cpu(), rc)
    near(probs, rp, 1.0 / E)
    near(loss[1], rl[1], 0.0)
    # p (cb (f - <p, f>) + 2 cz lse) / n: through autograd of logsumexp even 64 bits lose p where |x| > 1e16
    p, f = softmax(clean(x)), rc.double() * E / (k * nt[0])
    lse = torch.logsumexp(clean(x), -1, keepdim=True)
    want = 1.5 / nt[0] * p * (cb * (f - (p * f).sum(-1, keepdim=True)) + 2 * cz * lse)
    gl = torch.tensor(1.5).cuda()
    got = ep.balance_loss_backward(gl, x.cuda(), counts, k, balance_coef=cb, z_coef=cz)
    near(got, want, largest(want, E * cb * 1.5 / nt[0]), dtype)
    for score, renorm, scale in OPTIONS:         # and with the weights' gradient in the same pass
        alone = ep.route_backward(gw.cuda(), x.cuda(), idx.cuda(), score=score, renormalize=renorm, scale=scale)
        both = ep.route_backward(gw.cuda(), x.cuda(), idx.cuda(), score=score, renormalize=renorm, scale=scale,
                                 grad_loss=gl, counts=counts, balance_coef=cb, z_coef=cz)
        assert torch.isfinite(both).all()
        if dtype == torch.float32:
            total = want + alone.cpu().double()
            near(both, total, largest(total, E * cb + 4 * scale * float(gw.abs().max())))
    few = large_rows(E, dtype, 1e10)             # z, where its squares fit 32 bits
    i = idx[:, :few.shape[1]].contiguous()
    loss, _, _ = ep.balance_loss(few.cuda(), i.cuda(), balance_coef=cb, z_coef=cz)
    near(loss, ref_loss(clean(few), i, [few.shape[1]], cb, cz)[0], 0.0)


@pytest.mark.parametrize("W,T,E,k", [(1, 6, 8, 2), (2, 40, 77, 3), (4, 3000, 64, 4)])
def test_without_the_z_loss_its_size_does_not_matter(W, T, E, k):
    """One token whose whole row is at the type's lowest number: the square of
    its log-sum-exp is past fp32, and with z_coef 0 it has no part in the total."""
    for dtype in (torch.float32, torch.bfloat16):
        x = draw_logits(W, T, E, dtype, seed=E)
        x[0, 3] = torch.finfo(dtype).min
        idx = torch.argsort(torch.rand((W, T, E), generator=torch.Generator().manual_seed(T)), -1)[..., :k]
        idx = idx.to(torch.int32).contiguous()
        nt = [T] * W
        rl, rc, rp = ref_loss(clean(x), idx, nt, 0.5, 0.0)
        loss, counts, probs = ep.balance_loss(x.cuda(), idx.cuda(), balance_coef=0.5, z_coef=0.0)
        near(loss[:2], rl[:2], 0.0)
        near(probs, rp, 1.0 / E)
        assert torch.equal(counts.cpu(), rc)


@pytest.mark.parametrize("E,k", [(8, 2), (8, 1), (77, 3), (256, 8), (257, 32), (600, 6)])
def test_renormalised_sigmoid_of_very_low_logits(E, k):
    """Scores below what fp32 holds still have ratios: weights that sum to the
    scale, and gradients, as in 64 bits.  A weight's relative error is that of
    a difference of logits, 2^-23 of up to 10 and of the logit's own size."""
    rows = 64
    g = torch.Generator().manual_seed(E)
    level = torch.linspace(-30.0, -690.0, rows, dtype=torch.float64)
    level[:8] = torch.tensor([-80.0, -86.0, -87.4, -88.0, -88.5, -88.8, -95.0, -103.0])
    x = level[:, None] + torch.rand((rows, E), generator=g, dtype=torch.float64) * 5.0
    x[-6:] = torch.tensor([-2.0, 3.0, -90.0, -60.0, -50.0, -45.0])[:, None] - torch.arange(E) * 7.0    # few of a row low
    x[-8, 1:] = -math.inf
    x[-7] = -math.inf
    for dtype in DTYPES:
        xt = x.to(dtype)[None]
        w, idx = ep.route(xt.cuda(), k, score="sigmoid", scale=2.5)
        rw, ridx = ref_route(xt, k, "sigmoid", True, 2.5, None, [rows])
        assert torch.equal(idx.cpu(), ridx)
        near(w, rw, 2.5)
        gw = torch.randn((1, rows, k), generator=g)
        xs = clean(xt).requires_grad_(True)
        want, = torch.autograd.grad((weights_of(xs, ridx.long(), "sigmoid", True, 2.5) * gw).sum(), xs)
        got = ep.route_backward(gw.cuda(), xt.cuda(), idx, score="sigmoid", scale=2.5)
        assert torch.isfinite(got).all()
        near(got, torch.nan_to_num(want, nan=0.0), 4 * 2.5 * float(gw.abs().max()), dtype)


def test_defaults_of_the_losses_agree():
    """The combined gradient's loss is balance_loss's own unless told otherwise."""
    x = draw_logits(2, 30, 24, torch.float32, seed=8).cuda()
    w, idx = ep.route(x, 4)
    loss, counts, _ = ep.balance_loss(x, idx)
    gw, gl = torch.randn_like(w), torch.tensor(0.6).cuda()
    both = ep.route_backward(gw, x, idx, grad_loss=gl, counts=counts)
    parts = ep.route_backward(gw, x, idx) + ep.balance_loss_backward(gl, x, counts, 4)
    near(both, parts.cpu().double(), 4 * float(gw.abs().max()) + 24)
    assert (both - ep.route_backward(gw, x, idx)).abs().max() > 1e-4


@pytest.mark.parametrize("dtype", DTYPES)
def test_choice_by_score_plus_bias(dtype):
    """Scores in place of logits choose by score + bias; the gradient takes those indices."""
    W, T, E, k = 2, 50, 96, 6
    x = draw_logits(W, T, E, dtype, seed=12).cuda()
    bias = (torch.randn(E, generator=torch.Generator().manual_seed(2)) * 0.1).cuda()
    s = torch.sigmoid(x.float())
    _, idx = ep.route(s, k, bias=bias)
    want = torch.sort(s.cpu() + bias.cpu(), dim=-1, descending=True, stable=True).indices[..., :k]
    assert torch.equal(idx.cpu().long(), want)
    assert not torch.equal(ep.route(x, k, bias=bias)[1], idx)
    gw = torch.randn((W, T, k)).cuda()
    xs = clean(x.cpu()).requires_grad_(True)
    grad, = torch.autograd.grad((weights_of(xs, want, "sigmoid", True, 2.5) * gw.cpu()).sum(), xs)
    got = ep.route_backward(gw, x, idx, score="sigmoid", scale=2.5)
    near(got, grad, 4 * 2.5 * float(gw.abs().max()), dtype)
