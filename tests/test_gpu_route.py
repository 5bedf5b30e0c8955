"""Routing, balance loss and their gradients on the GPU against the formulas
in 64 bits.

Tolerances, fixed from the arithmetic: every output is a ratio or sum of a few
fp32 exponentials (each within a few 2^-24 relative, its argument's rounding
included: |x - max| below 40 where the result is not negligible), so 1e-5 of
the largest term bounds fp32 results; results in a 16-bit type add half a
unit in its last place."""
import math

import pytest
import torch

import combine_ep_layout_06_gb300 as ep

pytestmark = pytest.mark.gpu

UNIT = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -24}
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def draw_logits(W, T, E, dtype, seed=0, closed=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((W, T, E), generator=g) * 1.5
    if closed:
        x[torch.rand((W, T, E), generator=g) < closed] = -math.inf
    return x.to(dtype)


def clean(x):
    return torch.nan_to_num(x.double(), nan=-math.inf, posinf=torch.finfo(torch.float32).max, neginf=-math.inf)


def softmax(x):
    shut = (x == -math.inf).all(-1, keepdim=True)
    p = torch.softmax(torch.where(shut, torch.zeros_like(x), x), -1)
    return torch.where(shut, torch.zeros_like(p), p)


def weights_of(x, ids, score, renorm, scale):
    v = x.gather(-1, ids)
    if score == "softmax":
        v = softmax(v) if renorm else softmax(x).gather(-1, ids)
    else:
        v = torch.sigmoid(v)
        if renorm:
            s = v.sum(-1, keepdim=True)
            v = v / torch.where(s > 0, s, torch.ones_like(s))
    return v * scale


def ref_route(x, k, score, renorm, scale, bias, nt):
    key = clean(x).float()
    if bias is not None:
        key = key + bias
    ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :k]
    w = weights_of(clean(x), ids, score, renorm, scale)
    for s, n in enumerate(nt):
        ids[s, n:] = -1
        w[s, n:] = 0
    return w, ids.to(torch.int32)


def ref_loss(x, idx, nt, cb, cz):
    W, T, E = x.shape
    k = idx.shape[-1]
    n = sum(nt)
    counts = torch.zeros(E, dtype=torch.int64)
    share = torch.zeros(E, dtype=torch.float64)
    z = torch.zeros((), dtype=torch.float64)
    for s in range(W):
        rows, ids = x[s, :nt[s]], idx[s, :nt[s]].flatten().long()
        counts += torch.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
        share = share + softmax(rows).sum(0)
        lse = torch.logsumexp(rows, -1)
        z = z + torch.where(torch.isinf(lse), torch.zeros_like(lse), lse).square().sum()
    n = max(n, 1)
    balance = (counts.double() * E / (k * n) * share / n).sum()
    return torch.stack([cb * balance + cz * z / n, balance, z / n]), counts.to(torch.int32), share / n


def near(got, want, scale, dtype=torch.float32):
    got, want = got.cpu().double(), want.detach()
    tol = 1e-5 * scale + (UNIT[dtype] + 1e-5) * want.abs() + TINY[dtype]
    bad = (got - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), float((got - want).abs().max()))


SHAPES = [(1, 1, 1, 1), (1, 1, 8, 2), (2, 3, 9, 9), (3, 65, 77, 3), (8, 129, 8, 2), (2, 100, 256, 8),
          (1, 33, 257, 32), (4, 17, 1024, 6), (1, 70, 600, 1), (2, 40, 160, 16), (1, 9, 17, 5)]
OPTIONS = [("softmax", True, 1.0), ("softmax", False, 2.5), ("sigmoid", True, 2.5), ("sigmoid", False, 1.0)]


@pytest.mark.parametrize("W,T,E,k", SHAPES)
@pytest.mark.parametrize("score,renorm,scale", OPTIONS)
def test_route_and_its_gradient(W, T, E, k, score, renorm, scale):
    for i, dtype in enumerate(DTYPES):
        closed = 0.3 if i == 1 else 0.0
        x = draw_logits(W, T, E, dtype, seed=T + E + i, closed=closed)
        g = torch.Generator().manual_seed(E)
        bias = torch.randn(E, generator=g) * 0.3 if i != 2 else None
        nt = [T] * W if i == 0 else [max(0, T - 3 * s) for s in range(W)]
        w, idx = ep.route(x.cuda(), k, score=score, renormalize=renorm, scale=scale,
                          bias=None if bias is None else bias.cuda(), num_tokens=nt)
        rw, ridx = ref_route(x, k, score, renorm, scale, bias, nt)
        assert torch.equal(idx.cpu(), ridx)
        near(w, rw, scale)
        # gradient, with and without the balance loss in the same pass
        gw = torch.randn((W, T, k), generator=g)
        ids = ridx.long().clamp(min=0)
        counts = torch.randint(0, 50, (E,), generator=g, dtype=torch.int32)
        gl = torch.tensor(0.7)
        cb, cz, n = 0.5, 0.25, max(1, sum(nt))
        for loss in (False, True):
            xs = clean(x).requires_grad_(True)
            goal = torch.zeros((), dtype=torch.float64)
            for s in range(W):
                rows = xs[s, :nt[s]]
                seen = (rows.detach() > -math.inf).any(-1)
                rows = rows[seen]
                wt = weights_of(rows, ids[s, :nt[s]][seen], score, renorm, scale)
                goal = goal + (wt * gw[s, :nt[s]][seen]).sum()
                if loss:
                    f = counts.double() * E / (k * n)
                    goal = goal + gl.double() / n * (cb * (softmax(rows) * f).sum()
                                                     + cz * torch.logsumexp(rows, -1).square().sum())
            want, = torch.autograd.grad(goal, xs, allow_unused=True)
            want = torch.zeros_like(xs) if want is None else torch.nan_to_num(want, nan=0.0)
            extra = dict(grad_loss=gl.cuda(), counts=counts.cuda(), balance_coef=cb, z_coef=cz) if loss else {}
            got = ep.route_backward(gw.cuda(), x.cuda(), idx, score=score, renormalize=renorm, scale=scale,
                                    num_tokens=nt, **extra)
            assert got.dtype == dtype and got.shape == x.shape
            near(got, want, scale * float(gw.abs().max()) * (4 if k > 1 else 1) + (E if loss else 0), dtype)
    torch.cuda.synchronize()


@pytest.mark.parametrize("W,T,E,k", SHAPES + [(8, 700, 256, 8), (1, 5000, 8, 2)])
def test_balance_loss_and_its_gradient(W, T, E, k):
    for i, dtype in enumerate(DTYPES):
        x = draw_logits(W, T, E, dtype, seed=3 * T + E + i, closed=0.2 if i == 2 else 0.0)
        g = torch.Generator().manual_seed(T)
        idx = torch.argsort(torch.rand((W, T, E), generator=g), -1)[..., :k].to(torch.int32).contiguous()
        nt = [T] * W if i != 1 else [T // (s + 1) for s in range(W)]
        cb, cz = 0.5, 0.25
        loss, counts, probs = ep.balance_loss(x.cuda(), idx.cuda(), balance_coef=cb, z_coef=cz, num_tokens=nt)
        xs = clean(x).requires_grad_(True)
        rl, rc, rp = ref_loss(xs, idx, nt, cb, cz)
        assert torch.equal(counts.cpu(), rc)
        near(probs, rp, 1.0 / E)
        near(loss, rl, 0.0)
        again = ep.balance_loss(x.cuda(), idx.cuda(), balance_coef=cb, z_coef=cz, num_tokens=nt)
        assert all(torch.equal(a, b) for a, b in zip(again, (loss, counts, probs)))   # same bits each time
        want, = torch.autograd.grad(rl[0] * 1.5, xs)
        got = ep.balance_loss_backward(torch.tensor(1.5).cuda(), x.cuda(), counts, k, balance_coef=cb, z_coef=cz,
                                       num_tokens=nt)
        want = torch.nan_to_num(want, nan=0.0)
        near(got, want, float(want.abs().max()) + 1e-12, dtype)


def test_gradient_agrees_with_differences():
    """The kernels' own losses and weights, moved along a direction: the change
    over 2 h against the gradient's product with it.  fp32 rounding of the
    weighted sums (1e-6) over 2 h = 0.02 plus the h^2 term stay below 1e-3."""
    W, T, E, k = 1, 4, 12, 3
    x = draw_logits(W, T, E, torch.float32, seed=5).cuda()
    v = torch.randn_like(x)
    gw = torch.randn((W, T, k)).cuda()
    h = 1e-2
    _, idx = ep.route(x, k)
    for score, renorm in [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)]:
        def value(y):
            w, i = ep.route(y, E, score=score, renormalize=False)
            order = torch.argsort(i, -1)                       # every expert's score, by id
            full = torch.gather(w, -1, order).gather(-1, idx.long())
            if renorm:
                full = full / full.sum(-1, keepdim=True)
            return float((full.double() * gw.double()).sum())
        d = ep.route_backward(gw, x, idx, score=score, renormalize=renorm)
        slope = (value(x + h * v) - value(x - h * v)) / (2 * h)
        assert abs(slope - float((d.double() * v.double()).sum())) < 1e-3 * max(1.0, abs(slope))
    loss, counts, _ = ep.balance_loss(x, idx, z_coef=0.5)
    d = ep.balance_loss_backward(torch.ones((), device="cuda"), x, counts, k, z_coef=0.5)
    up = ep.balance_loss(x + h * v, idx, z_coef=0.5)[0][0]
    down = ep.balance_loss(x - h * v, idx, z_coef=0.5)[0][0]
    slope = float(up.double() - down.double()) / (2 * h)
    assert abs(slope - float((d.double() * v.double()).sum())) < 1e-3 * max(1.0, abs(slope))


@pytest.mark.parametrize("dtype", DTYPES)
def test_special_values(dtype):
    """-inf, NaN, +inf, the type's lowest number, ties, signed zeros."""
    low = torch.finfo(dtype).min
    inf, nan = math.inf, math.nan
    rows = [[-inf] * 6, [nan] * 6, [low] * 6, [0.0, -0.0, 0.0, -0.0, 0.0, -0.0], [inf, 1, inf, 2, -inf, nan],
            [1, 1, 1, 1, 2, 2], [low, -inf, 3, nan, low, 3], [-inf, -inf, -inf, 0.5, -inf, -inf], [inf, low, 0, 0, 0, 0]]
    x = torch.tensor(rows, dtype=dtype)[None]
    nt = [len(rows)]
    for score, renorm, scale in OPTIONS:
        for k in (1, 3, 6):
            w, idx = ep.route(x.cuda(), k, score=score, renormalize=renorm, scale=scale)
            rw, ridx = ref_route(x, k, score, renorm, scale, None, nt)
            assert torch.equal(idx.cpu(), ridx)
            assert torch.isfinite(w).all()
            near(w, rw, scale)
            d = ep.route_backward(torch.ones_like(w), x.cuda(), idx, score=score, renormalize=renorm, scale=scale)
            assert torch.isfinite(d).all()
            assert (d[0, :2] == 0).all()                   # rows that see no expert
    finite = torch.tensor([r for r in rows if inf not in r and low not in r], dtype=dtype)[None]
    idx = torch.zeros((1, finite.shape[1], 2), dtype=torch.int32)
    loss, counts, probs = ep.balance_loss(finite.cuda(), idx.cuda(), z_coef=1.0)
    rl, rc, rp = ref_loss(clean(finite), idx, [finite.shape[1]], 1.0, 1.0)
    assert torch.equal(counts.cpu(), rc)
    near(loss, rl, 0.0)
    near(probs, rp, 1.0)
    assert ep.moe_error() == 0


def test_strided_logits_streams_and_no_tokens():
    big = draw_logits(2, 50, 300, torch.bfloat16, seed=9).cuda()
    x = big[:, ::2, 3:260]
    w, idx = ep.route(x, 8, bias=None)
    w2, idx2 = ep.route(x.contiguous(), 8)
    assert torch.equal(w, w2) and torch.equal(idx, idx2)
    d = ep.route_backward(torch.ones_like(w), x, idx, renormalize=False)
    assert torch.equal(d, ep.route_backward(torch.ones_like(w), x.contiguous(), idx, renormalize=False))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    w3, idx3 = ep.route(x, 8, stream=side)
    loss3 = ep.balance_loss(x, idx3, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(w, w3) and torch.equal(idx, idx3)
    assert all(torch.equal(a, b) for a, b in zip(loss3, ep.balance_loss(x, idx)))
    # 2-D logits are one rank's
    w4, idx4 = ep.route(x[1], 8)
    assert torch.equal(w[1], w4) and torch.equal(idx[1], idx4)
    # nobody is there
    w, idx = ep.route(x, 8, num_tokens=[0, 0])
    assert (w == 0).all() and (idx == -1).all()
    loss, counts, probs = ep.balance_loss(x, idx2, num_tokens=[0, 0], z_coef=1.0)
    assert (loss == 0).all() and (counts == 0).all() and (probs == 0).all()
    d = ep.balance_loss_backward(torch.ones((), device="cuda"), x, counts, 8, num_tokens=[0, 0], z_coef=1.0)
    assert (d == 0).all()
    w, idx = ep.route(x[:, :0], 8)
    assert w.shape == (2, 0, 8) and idx.shape == (2, 0, 8)


def test_offsets_past_32_bits_and_graph_replay():
    gap = 1 << 31
    x = draw_logits(2, 40, 64, torch.bfloat16, seed=21).cuda()
    big = torch.empty(gap + x[1].numel(), dtype=x.dtype, device="cuda")
    far = torch.as_strided(big, x.shape, (gap, 64, 1))
    far.copy_(x)
    w, idx = ep.route(x, 6)
    assert all(torch.equal(a, b) for a, b in zip(ep.route(far, 6), (w, idx)))
    loss = ep.balance_loss(x, idx, z_coef=0.1)
    assert all(torch.equal(a, b) for a, b in zip(ep.balance_loss(far, idx, z_coef=0.1), loss))
    one = torch.ones((), device="cuda")
    d = ep.route_backward(w, x, idx, grad_loss=one, counts=loss[1], balance_coef=1.0, z_coef=0.1)
    assert torch.equal(ep.route_backward(w, far, idx, grad_loss=one, counts=loss[1], balance_coef=1.0, z_coef=0.1), d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w2, idx2 = ep.route(x, 6)
        loss2 = ep.balance_loss(x, idx2, z_coef=0.1)
        d2 = ep.route_backward(w2, x, idx2, grad_loss=one, counts=loss2[1], balance_coef=1.0, z_coef=0.1)
    for _ in range(2):
        d2.zero_()
        graph.replay()
        assert torch.equal(w, w2) and torch.equal(idx, idx2) and torch.equal(d, d2)
        assert all(torch.equal(a, b) for a, b in zip(loss, loss2))


def test_ids_out_of_range_are_skipped_and_reported():
    x = draw_logits(1, 5, 20, torch.float32, seed=2).cuda()
    w, idx = ep.route(x, 4)
    bad = idx.clone()
    bad[0, 2, 1] = 20
    bad[0, 3, 0] = -5
    assert ep.moe_error() == 0
    _, counts, _ = ep.balance_loss(x, bad)
    assert int(counts.sum()) == 5 * 4 - 2
    assert ep.moe_error() == 1 and ep.moe_error() == 0
    d = ep.route_backward(torch.ones_like(w), x, bad)
    assert torch.isfinite(d).all() and ep.moe_error() == 1


def test_routes_dispatch_as_it_takes_them():
    """route's outputs go into dispatch as they are."""
    W, T, E, k, H = 2, 40, 8, 2, 256
    x = draw_logits(W, T, E, torch.bfloat16, seed=4).cuda()
    w, idx = ep.route(x, k)
    op = ep.EpDispatchCombineOp(ep.EpDispatchCombineConfig(W, E, k, H, T))
    h = torch.randn((W, T, H)).to(torch.bfloat16).cuda()
    op.dispatch(h, w, None, idx)
    op.identity_expert()
    out, _ = op.combine()
    torch.cuda.synchronize()
    assert op.get_error() == (0, 0)
    # the identity expert weighs a row per rank in bf16: two roundings of parts that sum to h
    assert ((out.double() - h.double()).abs() <= 2.0 ** -7 * h.double().abs() + 1e-6).all()
