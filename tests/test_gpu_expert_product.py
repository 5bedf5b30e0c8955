"""Expert products and their gradients on the GPU against the formula in 64
bits.

Tolerances, fixed from the arithmetic.  u is half a unit in the last place
of the type (2^-8 bf16, 2^-11 fp16).  A sum of K products in fp32 is within
K * 2^-23 of the sum of the products' magnitudes; activations have slopes
below 1.13; outputs are rounded once, and the gradients' d = grad * act'(pre)
once before their products."""
import pytest
import torch

import combine_ep_layout_06_gb300 as ep

pytestmark = pytest.mark.gpu

U = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16)}
SMALL = {torch.bfloat16: 1e-30, torch.float16: 2.0 ** -24}


def act(name, v):
    if name == "swiglu":
        n = v.shape[-1] // 2
        return torch.nn.functional.silu(v[:, :n]) * v[:, n:]
    return {"none": lambda t: t * 1.0, "relu": torch.relu, "silu": torch.nn.functional.silu,
            "gelu": torch.nn.functional.gelu}[name](v)


def layout(R, counts, gap=0):
    """Offsets of groups that follow one another with `gap` rows between."""
    off = []
    for row in counts:
        run, o = 0, []
        for c in row:
            o.append(run)
            run += c + gap
        off.append(o)
    return off


def make(R, per, counts, K, N, dtype, name, seed=0, gap=0, rows=None, spoil=False):
    g = torch.Generator().manual_seed(seed)
    wide = 2 * N if name == "swiglu" else N
    offsets = layout(R, counts, gap)
    need = max(o[-1] + c[-1] for o, c in zip(offsets, counts)) if per else 0
    rows = max(1, need) if rows is None else rows

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g) * std).to(dtype)

    d = dict(x=normal(R, rows, K), weight=normal(R * per, wide, K, std=K ** -0.5), bias=normal(R * per, wide, std=0.3),
             residual=normal(R, rows, N), pre=normal(R, rows, wide), grad=normal(R, rows, N, std=0.2),
             count=torch.tensor(counts, dtype=torch.int32), offset=torch.tensor(offsets, dtype=torch.int32))
    if spoil:            # what lies outside every group must not matter
        used = torch.zeros((R, rows), dtype=torch.bool)
        for r in range(R):
            for o, c in zip(offsets[r], counts[r]):
                used[r, o:o + c] = True
        for n in ("x", "residual", "pre", "grad"):
            d[n][~used] = float("nan")
    return d, wide, rows


def groups(d, rows):
    R, per = d["count"].shape
    for r in range(R):
        for e in range(per):
            o, c = int(d["offset"][r, e]), int(d["count"][r, e])
            if c <= 0 or o < 0 or o >= rows:
                c = 0
            yield r * per + e, r, slice(o, min(o + c, rows)) if c else slice(0, 0)


def check(d, K, N, wide, rows, dtype, name, bias=True, residual=True, backward=True, views=lambda t: t, stream=None):
    dev = {n: views(t.cuda()) if t.is_floating_point() and n != "bias" else t.cuda() for n, t in d.items()}
    R = d["x"].shape[0]
    mark = 77.0
    out = torch.full((R, rows, N), mark, dtype=dtype, device="cuda")
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    y, pre = ep.expert_product(dev["x"], dev["weight"], dev["count"], dev["offset"],
                               bias=dev["bias"] if bias else None, activation=name,
                               residual=dev["residual"] if residual else None, save_pre=True, out=out, stream=stream)
    if backward:
        dx, dw, db = ep.expert_product_backward(dev["grad"], dev["x"], dev["weight"], dev["count"], dev["offset"],
                                                pre=dev["pre"], activation=name, bias_grad=bias, stream=stream)
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    assert y is out and ep.moe_error() == 0
    u, small = U[dtype], SMALL[dtype]
    y, pre = y.cpu().double(), pre.cpu().double()
    touched = torch.zeros((R, rows), dtype=torch.bool)
    for g, r, s in groups(d, rows):
        touched[r, s] = True
        x, w = d["x"][r, s].double(), d["weight"][g].double()
        b = d["bias"][g].double() if bias else torch.zeros(wide, dtype=torch.float64)
        v = x @ w.T + b
        e = (K + 4) * 2.0 ** -23 * (x.abs() @ w.abs().T + b.abs())
        assert ((pre[r, s] - v).abs() <= u * v.abs() + 1.01 * e + small).all(), g
        want, slope = act(name, v), 1.13 * e + 2e-6 * v.abs()
        if name == "swiglu":
            gate, up = v[:, :N], v[:, N:]
            slope = ((1.13 * e[:, :N] + 2e-6 * gate.abs()) * (up.abs() + e[:, N:])
                     + (gate.abs() + 0.3) * (e[:, N:] + 2e-6 * up.abs()))
        if residual:
            want = want + d["residual"][r, s].double()
        assert ((y[r, s] - want).abs() <= 1.01 * (u * want.abs() + slope) + small).all(), g
        if not backward:
            continue
        p = d["pre"][r, s].double().requires_grad_(True)
        dd, = torch.autograd.grad(act(name, p), p, d["grad"][r, s].double())
        rnd = u + 8e-6                                  # d's rounding and its fp32 arithmetic
        # where act' comes from cancelling terms (gelu, silu below 0) its error is 4e-6 of the gradient
        off = 4e-6 * (d["grad"][r, s].double().abs() * (1 + (p.detach().abs() if name != "swiglu" else 0)) if name != "swiglu"
                      else torch.cat([d["grad"][r, s].double().abs()] * 2, -1) * (1 + p.detach().abs()) * (1 + p.detach().abs().roll(N, -1)))
        da = rnd * dd.abs() + off + small
        want = dd @ w
        tol = u * want.abs() + da @ w.abs() + (wide + 4) * 2.0 ** -23 * (dd.abs() @ w.abs())
        assert ((dx[r, s].cpu().double() - want).abs() <= 1.01 * tol + small).all(), g
        want, n = dd.T @ x, x.shape[0]
        tol = u * want.abs() + da.T @ x.abs() + (n + 4) * 2.0 ** -23 * (dd.abs().T @ x.abs())
        assert ((dw[g].cpu().double() - want).abs() <= 1.01 * tol + small).all(), g
        if bias:
            want = dd.sum(0)
            tol = u * want.abs() + off.sum(0) + (n + 8) * 2.0 ** -23 * dd.abs().sum(0) + 8e-6 * dd.abs().sum(0)
            assert ((db[g].cpu().double() - want).abs() <= 1.01 * tol + small).all(), g
    assert (y[~touched] == mark).all()


CASES = [
    # R, counts per group, K, N
    (1, [[1]], 8, 8),
    (1, [[1]], 64, 128),
    (1, [[5]], 72, 136),
    (1, [[0, 1, 0, 2]], 256, 512),
    (2, [[3, 0, 17, 1], [0, 0, 40, 16]], 200, 328),
    (1, [[128]], 512, 256),
    (1, [[129, 255, 256, 257]], 192, 264),
    (1, [[700]], 1032, 776),
    (3, [[31, 33], [0, 0], [64, 1]], 320, 1000),
    (1, [[7] * 40], 128, 72),
    (1, [[2000, 0, 3]], 264, 1544),
]


@pytest.mark.parametrize("R,counts,K,N", CASES)
@pytest.mark.parametrize("name", ["none", "relu", "gelu", "silu", "swiglu"])
def test_products_and_gradients(R, counts, K, N, name):
    dtype = torch.float16 if (K // 8 + len(name)) % 2 else torch.bfloat16
    d, wide, rows = make(R, len(counts[0]), counts, K, N, dtype, name, seed=K + N)
    check(d, K, N, wide, rows, dtype, name)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("name", ["none", "swiglu"])
def test_rows_outside_the_groups_do_not_matter(dtype, name):
    """NaN between the groups reaches no output, and those rows of `out` stay."""
    d, wide, rows = make(2, 3, [[5, 70, 0], [1, 130, 19]], 136, 200, dtype, name, seed=1, gap=3, rows=300, spoil=True)
    check(d, 136, 200, wide, rows, dtype, name)
    check(d, 136, 200, wide, rows, dtype, name, bias=False, residual=False)


def test_counts_past_the_segment_are_cut():
    """count and offset as an overflowing grouping leaves them."""
    d, wide, rows = make(1, 4, [[20, 30, 40, 50]], 64, 64, torch.bfloat16, "silu", seed=2, rows=75)
    check(d, 64, 64, wide, rows, torch.bfloat16, "silu")
    d["count"][0, 0] = -3
    d["offset"][0, 1] = -1
    check(d, 64, 64, wide, rows, torch.bfloat16, "silu")


def test_strided_tensors_and_another_stream():
    def views(t):          # rows 40 elements further apart, segments too
        if t.dim() != 3:
            return t
        big = torch.full((t.shape[0], t.shape[1] + 5, t.shape[2] + 40), float("nan"), dtype=t.dtype, device=t.device)
        v = big[:, 2:2 + t.shape[1], 16:16 + t.shape[2]]
        v.copy_(t)
        return v
    d, wide, rows = make(2, 2, [[50, 9], [0, 77]], 128, 136, torch.float16, "swiglu", seed=3)
    check(d, 128, 136, wide, rows, torch.float16, "swiglu", views=views, stream=torch.cuda.Stream())


def test_offsets_past_32_bits():
    """Segments 2^31 elements apart: every tensor's last segment ends beyond
    what 32 bits of elements (or of bytes) reach."""
    gap = 1 << 31
    R, rows, K, N = 2, 70, 64, 72
    d, wide, rows = make(R, 2, [[30, 40], [9, 61]], K, N, torch.bfloat16, "silu", seed=11, rows=rows)

    def far(t):
        big = torch.empty(gap + t[1].numel(), dtype=t.dtype, device="cuda")
        v = torch.as_strided(big, t.shape, (gap, t.shape[2], 1))
        v.copy_(t)
        return v
    x, res, out = far(d["x"]), far(d["residual"]), far(torch.zeros((R, rows, N), dtype=torch.bfloat16))
    a = {n: t.cuda() for n, t in d.items()}
    y = ep.expert_product(x, a["weight"], a["count"], a["offset"], activation="silu", residual=res, out=out)
    want = ep.expert_product(a["x"], a["weight"], a["count"], a["offset"], activation="silu", residual=a["residual"])
    assert torch.equal(y, want)
    del res, out, y
    pre, grad = far(d["pre"]), far(d["grad"])
    got = ep.expert_product_backward(grad, x, a["weight"], a["count"], a["offset"], pre=pre, activation="silu", bias_grad=True)
    want = ep.expert_product_backward(a["grad"], a["x"], a["weight"], a["count"], a["offset"], pre=a["pre"],
                                      activation="silu", bias_grad=True)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_residual_in_place_and_graph_replay():
    """out may be the residual itself; a captured call replays."""
    d, wide, rows = make(1, 3, [[100, 0, 57]], 256, 320, torch.bfloat16, "gelu", seed=12)
    a = {n: t.cuda() for n, t in d.items()}
    args = (a["x"], a["weight"], a["count"], a["offset"])
    want = ep.expert_product(*args, activation="gelu", residual=a["residual"])
    same = a["residual"].clone()
    assert ep.expert_product(*args, activation="gelu", residual=same, out=same) is same
    assert torch.equal(same, want)
    grads = ep.expert_product_backward(a["grad"], *args, pre=a["pre"], activation="gelu", bias_grad=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ep.expert_product(*args, activation="gelu", residual=a["residual"])
        g = ep.expert_product_backward(a["grad"], *args, pre=a["pre"], activation="gelu", bias_grad=True)
    for _ in range(2):
        y.zero_()
        graph.replay()
        assert torch.equal(y, want) and all(torch.equal(p, q) for p, q in zip(g, grads))


def test_many_small_groups():
    """More groups than the tile walk looks at in one go, most of them empty."""
    g = torch.Generator().manual_seed(13)
    counts = [[int(c) for c in torch.randint(0, 4, (150,), generator=g) * (torch.rand(150, generator=g) < 0.4)]
              for _ in range(2)]
    d, wide, rows = make(2, 150, counts, 64, 72, torch.bfloat16, "swiglu", seed=14)
    check(d, 64, 72, wide, rows, torch.bfloat16, "swiglu")


def test_one_group_of_all_rows():
    """No count and offset: a plain product, 2-D rows."""
    d, wide, rows = make(1, 1, [[333]], 264, 392, torch.bfloat16, "gelu", seed=4)
    x, w, b = d["x"][0].cuda(), d["weight"].cuda(), d["bias"].cuda()
    y = ep.expert_product(x, w, bias=b, activation="gelu")
    y2 = ep.expert_product(d["x"].cuda(), w, d["count"].cuda(), d["offset"].cuda(), bias=b, activation="gelu")
    assert y.shape == (333, 392) and torch.equal(y, y2[0])
    dx, dw, db = ep.expert_product_backward(d["grad"][0].cuda(), x, w, pre=d["pre"][0].cuda(), activation="gelu")
    assert dx.shape == x.shape and dw.shape == w.shape and db is None


def test_gradient_parts_can_be_left_out():
    """The C entry with grad_x or grad_w NULL gives the same other parts."""
    import ctypes

    from combine_ep_layout_06_gb300 import _lib
    d, wide, rows = make(1, 3, [[70, 0, 131]], 72, 136, torch.bfloat16, "silu", seed=15)
    a = {n: t.cuda() for n, t in d.items()}
    dx, dw, db = ep.expert_product_backward(a["grad"], a["x"], a["weight"], a["count"], a["offset"], pre=a["pre"],
                                            activation="silu", bias_grad=True)
    L = _lib.load()

    def r(t):
        return _lib.EpRowsC(t.data_ptr() if t is not None else None, 0, t.shape[-1] if t is not None else 0)
    desc = _lib.EpProductDescC(1, 3, rows, 72, 136, _lib.EP_DT_BF16, 3, 0, a["count"].data_ptr(),
                               a["offset"].data_ptr(), _lib.EpRowsC(a["weight"].data_ptr(), wide * 72, 72), r(a["x"]))
    need = ctypes.c_size_t(0)
    assert L.ep_expert_product_workspace(ctypes.byref(desc), ctypes.byref(need)) == 0
    scratch = torch.empty(need.value, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for want_x, want_w, want_b in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 1)):
        x2, w2, b2 = (torch.zeros_like(t) if on else None for t, on in ((dx, want_x), (dw, want_w), (db, want_b)))
        assert L.ep_expert_product_backward(
            ctypes.byref(desc), ctypes.byref(r(a["grad"])), ctypes.byref(r(a["pre"])), ctypes.byref(r(x2)),
            w2.data_ptr() if want_w else None, b2.data_ptr() if want_b else None, scratch.data_ptr(), need.value,
            None, stream) == 0
        for got, want in ((x2, dx), (w2, dw), (b2, db)):
            assert got is None or torch.equal(got, want)


def test_no_rows():
    w = torch.randn((3, 64, 32)).to(torch.bfloat16).cuda()
    x = torch.empty((1, 0, 32), dtype=torch.bfloat16, device="cuda")
    z = torch.zeros((1, 3), dtype=torch.int32, device="cuda")
    assert ep.expert_product(x, w, z, z).shape == (1, 0, 64)
    dx, dw, db = ep.expert_product_backward(torch.empty((1, 0, 64), dtype=torch.bfloat16, device="cuda"), x, w, z, z,
                                            bias_grad=True)
    assert dx.shape == x.shape and (dw == 0).all() and (db == 0).all()


def test_the_same_call_gives_the_same_bits():
    d, wide, rows = make(1, 8, [[300, 1, 0, 77, 1000, 12, 64, 500]], 512, 384, torch.bfloat16, "swiglu", seed=6)
    a = {n: t.cuda() for n, t in d.items()}
    runs = [(*ep.expert_product(a["x"], a["weight"], a["count"], a["offset"], bias=a["bias"], activation="swiglu",
                                save_pre=True),
             *ep.expert_product_backward(a["grad"], a["x"], a["weight"], a["count"], a["offset"], pre=a["pre"],
                                         activation="swiglu", bias_grad=True)) for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(runs[0], r))


def test_gradient_agrees_with_differences():
    """L = sum(y * c) moved along a direction of x: fp16 y with |y| of order 1
    is off by 2^-11 each, averaged over 64 x 48 outputs weighted by c; the step
    h = 2^-3 is exact in fp16 for the direction's values (+-1/2)."""
    g = torch.Generator().manual_seed(8)
    x = (torch.randint(-8, 9, (64, 40), generator=g) / 8).half()
    v = (torch.randint(0, 2, (64, 40), generator=g) - 0.5).half()
    w = (torch.randn((1, 96, 40), generator=g) * 0.1).half().cuda()
    c = torch.randn((64, 48), generator=g).half().cuda()
    h = 2.0 ** -3
    y, pre = ep.expert_product(x.cuda(), w, activation="swiglu", save_pre=True)
    dx, _, _ = ep.expert_product_backward(c, x.cuda(), w, pre=pre, activation="swiglu")
    up = ep.expert_product((x + h * v).cuda(), w, activation="swiglu").double()
    down = ep.expert_product((x - h * v).cuda(), w, activation="swiglu").double()
    slope = float(((up - down) * c.double()).sum()) / (2 * h)
    got = float((dx.cpu().double() * v.double()).sum())
    # rounding: 2 * 2^-11 * |y| * |c| summed in quadrature over the outputs, / (2 h); cubic term h^2 / 6 * third derivative
    noise = 4 * 2.0 ** -12 * float((y.double().abs() * c.double().abs()).square().sum().sqrt()) / (2 * h)
    assert abs(slope - got) <= noise + 2e-3 * max(1.0, float((dx.double().abs().sum() * 0.5) ** 0.5))
