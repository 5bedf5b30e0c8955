"""The experts of a few tokens against 64 bits.

Tolerance.  Sums are fp32, activations between the products are exact to 2^-16 of
their value (fp32, or two 16-bit halves), and out is rounded once: finfo.eps / 2 of each
value, and 2^-14 of the sum of magnitudes |w| |down| (|x| |up|) (at most 2^10 terms of
2^-24 each for both products, and the activation's few units)."""
import math

import pytest
import torch

import combine_ep_layout_06_gb300 as ep
from combine_ep_layout_06_gb300 import _lib

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def make(T, E, k, H, F, act="swiglu", dtype=BF, bias=False, residual=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)
    wide = 2 * F if act == "swiglu" else F
    c = dict(x=rand(T, H), up=rand(E, wide, H, std=H ** -0.5), down=rand(E, H, F, std=F ** -0.5), activation=act,
             up_bias=rand(E, wide, std=0.2) if bias else None, down_bias=rand(E, H, std=0.2) if bias else None,
             residual=rand(T, H) if residual else None)
    c["weights"] = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), -1)
    c["indices"] = torch.rand((T, E), generator=g, device="cuda").argsort(-1)[:, :k].to(torch.int32).contiguous()
    return c


# Layers of both kinds: little work (up to 48 MB of weights over all choices)
# and the kernels on tensor cores.
LAYERS = [(128, 64), (1032, 520)]


def call(c, **kw):
    return ep.moe_few_tokens(c["x"], c["weights"], c["indices"], c["up"], c["down"], activation=c["activation"],
                             up_bias=c["up_bias"], down_bias=c["down_bias"], residual=c["residual"], **kw)


def activation(v, name):
    f = torch.nn.functional
    if name == "swiglu":
        return f.silu(v.chunk(2, -1)[0]) * v.chunk(2, -1)[1]
    return {"none": lambda t: t, "relu": torch.relu, "gelu": f.gelu, "silu": f.silu}[name](v)


def reference(c):
    """out, and the sum of its terms' magnitudes."""
    x = c["x"].double()
    out = torch.zeros_like(x) if c["residual"] is None else c["residual"].double()
    size = out.abs()
    for t, ids in enumerate(c["indices"].tolist()):
        for j, e in enumerate(ids):
            if not 0 <= e < c["up"].shape[0]:
                continue
            up, down = c["up"][e].double(), c["down"][e].double()
            ub = 0 if c["up_bias"] is None else c["up_bias"][e].double()
            db = 0 if c["down_bias"] is None else c["down_bias"][e].double()
            w = float(c["weights"][t, j])
            out[t] += w * (down @ activation(up @ x[t] + ub, c["activation"]) + db)
            v = up.abs() @ x[t].abs() + (ub if c["up_bias"] is None else ub.abs())
            if c["activation"] == "swiglu":
                v = v.chunk(2, -1)[0] * v.chunk(2, -1)[1]
            size[t] += abs(w) * (down.abs() @ v + (db if c["down_bias"] is None else db.abs()))
    return out, size


def check(got, c):
    want, size = reference(c)
    eps = torch.finfo(got.dtype).eps
    off = (got.double() - want).abs()
    assert bool((off <= want.abs() * eps / 2 + size * 2.0 ** -14 + 2.0 ** -24).all()), float((off / (size + 1e-30)).max())
    # and over all: the rounding of out, with what is between the products far below it
    assert float(off.norm()) <= float(want.norm()) * (eps / 2 + 2.0 ** -13) + 1e-7
    assert ep.moe_error() == 0


@pytest.mark.parametrize("T,E,k,H,F", [
    (1, 1, 1, 8, 8), (1, 8, 2, 256, 192), (2, 3, 3, 64, 40), (3, 16, 4, 264, 136), (7, 40, 8, 512, 72), (8, 4, 1, 1024, 8),
    (9, 5, 5, 128, 1000), (16, 64, 6, 136, 128), (17, 300, 2, 72, 64), (31, 9, 9, 200, 88), (33, 2, 2, 640, 320), (64, 8, 2, 384, 256),
    (64, 1, 1, 264, 248), (64, 1024, 32, 16, 16), (5, 6, 2, 1000, 1000), (64, 1, 1, 776, 264), (64, 1024, 32, 72, 64),
    (63, 40, 30, 136, 40), (33, 33, 32, 8, 968), (34, 3, 3, 1024, 56), (1, 40, 32, 1000, 392), (48, 300, 8, 264, 72)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_against_the_formula(T, E, k, H, F, dtype):
    c = make(T, E, k, H, F, dtype=dtype, bias=T % 2 == 0, residual=T % 3 == 0, seed=T)
    check(call(c), c)


@pytest.mark.parametrize("T,E,k,H,F", [(17, 7, 1, 4168, 128), (6, 43, 3, 4000, 96), (64, 3, 1, 5000, 72), (33, 2, 2, 1032, 520)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_few_tiles_of_a_deep_product(T, E, k, H, F, dtype):
    """Sums of more than 2^10 terms: only the whole is compared."""
    c = make(T, E, k, H, F, dtype=dtype, bias=T % 2 == 0, residual=True, seed=T)
    c["indices"][0] = -1
    got, (want, _) = call(c), reference(c)
    assert float((got.double() - want).norm()) <= float(want.norm()) * (torch.finfo(dtype).eps / 2 + 2.0 ** -13)
    for _ in range(20):
        assert torch.equal(call(c), got)
    assert ep.moe_error() == 0


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu", "swiglu"])
@pytest.mark.parametrize("T,H,F", [(1, 320, 168), (20, 320, 168), (3, 1032, 776), (40, 520, 264), (20, 2056, 136)])
def test_activations(act, T, H, F):
    c = make(T, 6, 3, H, F, act=act, bias=True, residual=True, seed=5)
    check(call(c), c)


def test_wider_layers():
    """More than one slice of everything, and more work than SMs; magnitudes of
    2^10 terms no longer bound the sums, so only the whole is compared."""
    for T, E, k, H, F, act in ((1, 12, 8, 7168, 512, "swiglu"), (24, 12, 4, 2048, 1032, "swiglu"), (48, 4, 2, 4096, 328, "gelu")):
        c = make(T, E, k, H, F, act=act, seed=T)
        got, (want, _) = call(c), reference(c)
        assert float((got.double() - want).norm()) <= float(want.norm()) * (torch.finfo(BF).eps / 2 + 2.0 ** -13)


@pytest.mark.parametrize("H,F", LAYERS)
def test_absent_repeated_and_wrong_experts(H, F):
    c = make(9, 7, 4, H, F, bias=True, residual=True)
    idx = c["indices"]
    idx[0] = -1                                     # an absent token
    idx[1, 2:] = -1
    idx[2] = idx[2, 0]                              # one expert, four times
    idx[3, 1] = idx[3, 0]
    idx[4] = torch.tensor([-5, -1, 6, 0], device="cuda")
    got = call(c)
    check(got, c)
    assert torch.equal(got[0], c["residual"][0])
    c["residual"] = None
    assert bool((call(c)[0] == 0).all())
    idx[:] = -1
    assert bool((call(c) == 0).all())
    idx[5, 1], idx[6] = 7, 1 << 30                  # past the last expert: skipped and reported
    got = call(c)
    assert bool((got == 0).all()) and ep.moe_error() == _lib.EP_DEVERR_BAD_INDEX


@pytest.mark.parametrize("T", [9, 40, 64])
def test_an_expert_with_every_token(T):
    """More rows of one expert than an accumulator takes, next to experts of one."""
    c = make(T, 12, 3, 520, 392, bias=True)
    c["indices"][:, 1] = 5
    c["indices"][T // 2:, 2] = 5
    check(call(c), c)


@pytest.mark.parametrize("H,F", LAYERS)
def test_rows_do_not_meet(H, F):
    """NaN and infinities of one token, of an expert that nobody chose and of
    choices that are closed reach no other row."""
    c = make(12, 6, 2, H, F, residual=True)
    c["indices"][c["indices"] == 4] = 3
    clean = call(c)
    c["x"][5] = math.nan
    c["x"][6, 7] = math.inf
    c["up"][4], c["down"][4] = math.nan, math.inf
    c["weights"][7, 0], c["indices"][7, 0] = math.nan, -1
    c["indices"][8] = -1
    c["x"][8] = math.nan
    got = call(c)
    rest = torch.tensor([0, 1, 2, 3, 4, 9, 10, 11], device="cuda")
    assert torch.equal(got[rest], clean[rest])
    assert bool(got[5].isnan().all()) and bool(got[6].isnan().any()) and not bool(got[7].isnan().any())
    assert torch.equal(got[8], c["residual"][8])


@pytest.mark.parametrize("H,F", [(128, 64), (1032, 776)])
def test_activations_past_the_type(H, F):
    """Between the products values may pass what fp16 holds (up to 131008), and
    infinite ones stay infinite."""
    c = make(8, 4, 3, H, F, act="none", dtype=HF)
    c["up"] *= 100.0
    c["x"] *= 300.0
    c["down"] *= 2.0 ** -10
    v = torch.einsum("th,efh->tef", c["x"].double(), c["up"].double()).abs()
    c["x"] *= float(100000.0 / v.max())
    v = torch.einsum("th,efh->tef", c["x"].double(), c["up"].double()).abs()
    assert 65504 < float(v.max()) < 131008
    check(call(c), c)
    c["x"][3, 1] = math.inf
    got = call(c)
    assert not bool(got[3].isfinite().any()) and bool(got[torch.arange(8, device="cuda") != 3].isfinite().all())


@pytest.mark.parametrize("H,F", [(128, 64), (1032, 640)])
def test_layouts(H, F):
    """Ranks of tokens, strided rows and experts' slices of a larger tensor have the bits of dense ones."""
    c = make(6, 5, 2, H, F, residual=True)
    want = call(c)
    r = dict(c, x=c["x"].view(3, 2, H), residual=c["residual"].view(3, 2, H), weights=c["weights"].view(3, 2, 2),
             indices=c["indices"].view(3, 2, 2))
    assert torch.equal(call(r).view(6, H), want)
    wide = dict(c)
    for name, pad in (("x", 16), ("residual", 8), ("up", 24), ("down", 8)):
        t = c[name]
        big = torch.full(t.shape[:-1] + (t.shape[-1] + pad,), math.nan, dtype=t.dtype, device="cuda")
        big[..., :t.shape[-1]] = t
        wide[name] = big[..., :t.shape[-1]]
    assert torch.equal(call(wide), want)
    assert torch.equal(call(dict(c, up=c["up"].repeat(1, 2, 1)[:, :2 * F])), want)
    none = dict(c, x=c["x"][:0], residual=None, weights=c["weights"][:0], indices=c["indices"][:0])
    assert call(none).shape == (0, H)


def test_streams_graphs_and_two_at_once():
    cases = [make(T, 16, 4, 512, 256, seed=T, residual=True) for T in (1, 5, 40)]       # little work and tensor cores
    want = [call(c) for c in cases]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        got = [call(c, stream=s) for c, s in zip(cases, sides)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [call(c) for c in cases for _ in range(2)]
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for i, a in enumerate(got):
        assert torch.equal(a, want[i // 2])
    for c in cases:
        c["x"].neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], call(cases[0]))


@pytest.mark.parametrize("T,H,F", [(4, 256, 128), (12, 1024, 512)])
def test_a_chain_of_layers(T, H, F):
    """Each call starts while the one before it ends: every layer must see the
    last one's output."""
    layers = [make(T, 8, 2, H, F, seed=s) for s in range(6)]

    def chain(wait):
        x = layers[0]["x"]
        for c in layers * 5:
            x = call(dict(c, x=x, residual=x))
            x = ep.rms_norm(x, torch.ones(H, dtype=BF, device="cuda"))
            if wait:
                torch.cuda.synchronize()
        return x
    want = chain(True)
    for _ in range(5):
        assert torch.equal(chain(False), want)


def test_refusals():
    c = make(4, 4, 2, 64, 32)
    x, w, i, up, down = (c[n] for n in ("x", "weights", "indices", "up", "down"))
    for f in (lambda: ep.moe_few_tokens(x.float(), w, i, up.float(), down.float()), lambda: ep.moe_few_tokens(x, w, i, up.half(), down),
              lambda: ep.moe_few_tokens(x, w, i, up, down.half()), lambda: ep.moe_few_tokens(x, w, i.long(), up, down),
              lambda: ep.moe_few_tokens(x, w.half(), i, up, down), lambda: ep.moe_few_tokens(x, w[:2], i, up, down),
              lambda: ep.moe_few_tokens(x, w, i[:2], up, down), lambda: ep.moe_few_tokens(x, w, i, up[:3], down),
              lambda: ep.moe_few_tokens(x, w, i, up, down, activation="silu"), lambda: ep.moe_few_tokens(x, w, i, up, down, activation="mish"),
              lambda: ep.moe_few_tokens(x, w, i, up[..., :32], down), lambda: ep.moe_few_tokens(x.repeat(17, 1), w, i, up, down),
              lambda: ep.moe_few_tokens(x, w, i, up, down, residual=x[:2]), lambda: ep.moe_few_tokens(x, w, i, up, down, up_bias=x[:3]),
              lambda: ep.moe_few_tokens(x, w, i, up, down, down_bias=x.half()), lambda: ep.moe_few_tokens(x, w, i, up.cpu(), down),
              lambda: ep.moe_few_tokens(x[..., :60], w, i, up[..., :60], down[:, :60]), lambda: ep.moe_few_tokens(x, w[:, :0], i[:, :0], up, down),
              lambda: ep.moe_few_tokens(x.t(), w, i, up, down), lambda: ep.moe_few_tokens(x, w, i, up.transpose(1, 2), down)):
        with pytest.raises(ValueError):
            f()
    assert ep.moe_error() == 0
