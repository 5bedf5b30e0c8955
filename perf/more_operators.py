"""More operators of a mixture-of-experts layer, and the cases they are measured on.

rms_norm        root-mean-square norm with the residual's addition, in the rows' type or in 8 bits with scales, and its
                gradient
checkpoint      activations kept in 8 bits with scales: saved, restored through the activation, and taken by the
                expert product's gradient
moe_few_tokens  the experts of a few tokens, both products and the weighted sum

``own`` chooses between the plain forms below and the package's kernels.  8 bits are E4M3 codes with one fp32 scale
for every 128 values of a row: scale = max|v| / 448, code = v / scale rounded.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn
BLOCK = 128
SQRT2 = math.sqrt(2.0)
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # The norm of one decoded token with its residual: once or twice a layer, latency alone.
        dict(name="norm_one_token", op="norm", rows=1, width=7168, dtype="bf16", residual=True, eight=False),
        # The norm before a MoE layer in training or prefill, 8 ranks x 4096 tokens, as codes for an 8-bit dispatch.
        dict(name="norm_eight_batch", op="norm", rows=32768, width=7168, dtype="bf16", residual=True, eight=True),
        # The gradient for a small batch of odd rows, fp32.
        dict(name="norm_grad_odd", op="norm_backward", rows=333, width=1001, dtype="fp32", total=False),
        # The gradient in training, with what comes down the residual stream.
        dict(name="norm_grad_batch", op="norm_backward", rows=16384, width=7168, dtype="bf16", total=True),
        # Pre-activations of a rank's experts in training, put away in 8 bits.
        dict(name="checkpoint_save", op="save", ranks=2, groups=16, rows=32768, n=1792, dtype="bf16", act="swiglu", empty=1,
             layout=3),
        # Their activations again, as the down projection's gradient needs them.
        dict(name="checkpoint_restore", op="restore", ranks=2, groups=16, rows=32768, n=1792, dtype="bf16", act="swiglu",
             empty=1, layout=3),
        # The same of a small layer, odd rows, a part of a block at each row's end.
        dict(name="checkpoint_restore_small", op="restore", ranks=1, groups=8, rows=251, n=328, dtype="fp16", act="gelu",
             empty=2, layout=5),
        # The gradient of gate and up from pre-activations in 8 bits.
        dict(name="checkpoint_grad", op="grad", ranks=2, groups=8, rows=8192, n=1792, k=4096, dtype="bf16", act="swiglu",
             empty=1, layout=7),
        # A single stream's decode: one token, 8 of 256 experts.
        dict(name="few_one_token", op="few", tokens=1, experts=256, topk=8, hidden=7168, inner=1792, dtype="bf16",
             act="swiglu", bias=False, residual=True, absent=0, layout=11),
        # Decode of 16 streams over the same experts: about 100 of them are read.
        dict(name="few_16_tokens", op="few", tokens=16, experts=256, topk=8, hidden=7168, inner=1792, dtype="bf16",
             act="swiglu", bias=False, residual=False, absent=0, layout=13),
        # 64 streams over 8 experts of a wider layer, biases, some streams idle.
        dict(name="few_64_tokens", op="few", tokens=64, experts=8, topk=2, hidden=4096, inner=3584, dtype="fp16",
             act="swiglu", bias=True, residual=True, absent=5, layout=17),
        # A small model's layer: latency.
        dict(name="few_small", op="few", tokens=3, experts=8, topk=2, hidden=256, inner=192, dtype="bf16", act="gelu",
             bias=True, residual=False, absent=0, layout=19),
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "save", "restore", "grad", "few", "few", "few"])
    if op.startswith("norm"):
        case = dict(op=op, rows=spread(rng, 1, 32768), width=spread(rng, 64, 16384), dtype=rng.choice(["bf16", "fp16", "fp32"]))
        if op == "norm":
            case.update(residual=rng.random() < 0.5, eight=rng.random() < 0.5)
            if case["eight"]:
                case["width"] = BLOCK * spread(rng, 1, 112)
        else:
            case["total"] = rng.random() < 0.5
        while case["rows"] * case["width"] > 1 << 27:
            case["rows"] //= 2
        return case
    if op == "few":
        experts = spread(rng, 4, 256)
        case = dict(op=op, tokens=spread(rng, 1, 64), experts=experts, topk=rng.randint(1, min(8, experts)),
                    hidden=8 * spread(rng, 16, 896), inner=8 * spread(rng, 8, 448), dtype=rng.choice(["bf16", "fp16"]),
                    act=rng.choice(["swiglu", "swiglu", "gelu", "relu", "silu"]), bias=rng.random() < 0.4,
                    residual=rng.random() < 0.5, layout=rng.randrange(1 << 20))
        case["absent"] = rng.choice([0, 0, case["tokens"] // 4])
        while case["experts"] > case["topk"] and case["experts"] * case["hidden"] * case["inner"] > 1 << 30:
            case["experts"] -= 1
        return case
    ranks = rng.choice([1, 2])
    groups = ranks * spread(rng, 1, 16)
    case = dict(op=op, ranks=ranks, groups=groups, rows=ranks * spread(rng, 1, 8192), n=8 * spread(rng, 8, 256),
                dtype=rng.choice(["bf16", "fp16"]), act=rng.choice(["swiglu", "gelu", "silu", "relu"]),
                empty=rng.randint(0, (groups // ranks - 1) // 4), layout=rng.randrange(1 << 20))
    if op == "grad":
        case["k"] = 8 * spread(rng, 8, 512)
        while work(case)["flops"] > 4e11:
            case["rows"] = ranks * max(1, case["rows"] // ranks // 2)
    return case


def wide(case):
    """Features of the first product: gate and up where it is gated."""
    return case["n" if "n" in case else "inner"] * (2 if case["act"] == "swiglu" else 1)


def group_counts(case):
    """Rows of every group, from the case alone: uneven, `empty` groups of each rank without any."""
    rng = random.Random(case["layout"])
    per, rows = case["groups"] // case["ranks"], case["rows"] // case["ranks"]
    counts = []
    for _ in range(case["ranks"]):
        share = [rng.uniform(0.6, 1.4) for _ in range(per)]
        for g in rng.sample(range(per), min(case["empty"], per - 1)):
            share[g] = 0.0
        ends, run, total = [], 0.0, sum(share)
        for s in share:
            run += s
            ends.append(int(round(rows * run / total)))
        ends[-1] = rows
        counts += [b - a for a, b in zip([0] + ends[:-1], ends)]
    return counts


def choices(case):
    """Every token's experts, from the case alone; the last `absent` tokens have none."""
    rng = random.Random(case["layout"])
    here = case["tokens"] - case["absent"]
    return [rng.sample(range(case["experts"]), case["topk"]) if t < here else [-1] * case["topk"] for t in range(case["tokens"])]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, op = DTYPES[case["dtype"]], case["op"]

    def normal(*shape, std=1.0, dtype=dtype):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    def weights(n, rows, cols):
        w = torch.empty(n, rows, cols, dtype=dtype, device="cuda")
        for i in range(n):
            w[i] = normal(rows, cols, std=cols ** -0.5)
        return w

    s = dict(case=case)
    if op.startswith("norm"):
        rows, H = case["rows"], case["width"]
        s["weight"] = (torch.rand(H, generator=gen, device="cuda") + 0.5).to(dtype)
        s["x"] = normal(rows, H)
        if op == "norm":
            s["residual"] = normal(rows, H, std=2.0) if case["residual"] else None
        else:
            s["grad"] = normal(rows, H, std=0.1)
            s["grad_total"] = normal(rows, H, std=0.1) if case["total"] else None
    elif op == "few":
        T, E, H, F = case["tokens"], case["experts"], case["hidden"], case["inner"]
        s["x"], s["residual"] = normal(T, H), normal(T, H) if case["residual"] else None
        s["up"], s["down"] = weights(E, wide(case), H), weights(E, H, F)
        s["up_bias"] = normal(E, wide(case), std=0.1) if case["bias"] else None
        s["down_bias"] = normal(E, H, std=0.1) if case["bias"] else None
        s["indices"] = torch.tensor(choices(case), dtype=torch.int32, device="cuda")
        s["weights"] = torch.softmax(normal(T, case["topk"], dtype=torch.float32), -1) * (s["indices"] >= 0)
    else:
        R, G, n = case["ranks"], case["groups"], case["n"]
        cap, per, counts = case["rows"] // R, G // R, group_counts(case)
        offsets = [sum(counts[g - g % per:g]) for g in range(G)]
        s["count"] = torch.tensor(counts, dtype=torch.int32, device="cuda").view(R, per)
        s["offset"] = torch.tensor(offsets, dtype=torch.int32, device="cuda").view(R, per)
        s["pre"] = normal(R, cap, wide(case))
        if op != "save":
            s["codes"], s["scales"] = eight_bits(s.pop("pre").float())
        if op == "grad":
            # the plain form's padded layout: row i of group g stands at g * most + i
            most = max(counts)
            first = torch.tensor([g // per * cap + o for g, o in enumerate(offsets)], device="cuda")
            step = torch.arange(most, device="cuda")
            s["slots"] = (first[:, None] + step).clamp(max=R * cap - 1)
            s["here"] = step < torch.tensor(counts, device="cuda")[:, None]
            s["x"], s["grad"] = normal(R, cap, case["k"]), normal(R, cap, n, std=0.1)
            s["weight"] = weights(G, wide(case), case["k"])
    return s


# ------------------------------------------------------------ plain forms

def eight_bits(v):
    """Codes and scales of 32-bit rows: a block for every 128 values, the last one of a row perhaps a part."""
    width = v.shape[-1]
    blocks = -(-width // BLOCK)
    padded = torch.zeros(v.shape[:-1] + (blocks * BLOCK,), dtype=v.dtype, device=v.device)
    padded[..., :width] = v
    padded = padded.view(v.shape[:-1] + (blocks, BLOCK))
    scales = padded.abs().amax(-1) / 448.0
    q = padded / torch.where(scales > 0, scales, torch.ones_like(scales))[..., None]
    return q.flatten(-2)[..., :width].contiguous().to(E4M3), scales


def from_eight_bits(codes, scales):
    return codes.float() * scales.repeat_interleave(BLOCK, -1)[..., :codes.shape[-1]]


def activation(v, act, n):
    if act == "relu":
        return v.clamp(min=0)
    if act == "gelu":
        return v * 0.5 * (1.0 + torch.erf(v / SQRT2))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    return v[..., :n] / (1.0 + torch.exp(-v[..., :n])) * v[..., n:]


def plain_norm(s):
    case, total = s["case"], s["x"]
    if s["residual"] is not None:
        total = (total.float() + s["residual"].float()).to(total.dtype)
    h = total.float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    y = eight_bits(y) if case["eight"] else (y.to(total.dtype),)
    return y + (total,) if s["residual"] is not None else y


def plain_norm_backward(s):
    h, g = s["x"].float(), s["grad"].float()
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    u = g * s["weight"].float()
    dx = r * u - h * (r * r * r * (u * h).mean(-1, keepdim=True))
    if s["grad_total"] is not None:
        dx = dx + s["grad_total"].float()
    return dx.to(s["x"].dtype), (g * h * r).sum(0).to(s["weight"].dtype)


def plain_save(s):
    return eight_bits(s["pre"].float())


def plain_restore(s):
    case = s["case"]
    return activation(from_eight_bits(s["codes"], s["scales"]), case["act"], case["n"]).to(DTYPES[case["dtype"]])


def plain_grad(s):
    case, n, act = s["case"], s["case"]["n"], s["case"]["act"]

    def padded(t):
        t = t.reshape(-1, t.shape[-1])[s["slots"]]
        return torch.where(s["here"][..., None], t, torch.zeros_like(t))

    g, v, x = padded(s["grad"].float()), padded(from_eight_bits(s["codes"], s["scales"])), s["x"]
    if act == "relu":
        d = torch.where(v > 0, g, torch.zeros_like(g))
    elif act == "gelu":
        d = g * (0.5 * (1.0 + torch.erf(v / SQRT2)) + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi))
    else:
        gate = v[..., :n]
        sig = 1.0 / (1.0 + torch.exp(-gate))
        d = g * sig * (1.0 + gate * (1.0 - sig))
        if act == "swiglu":
            d = torch.cat([d * v[..., n:], g * gate * sig], -1)
    dx = torch.zeros_like(x).view(-1, x.shape[-1])
    dx[s["slots"][s["here"]]] = torch.bmm(d, s["weight"].float())[s["here"]].to(x.dtype)
    return dx.view(x.shape), torch.bmm(d.transpose(1, 2), padded(x.float())).to(x.dtype)


def plain_few(s):
    case, x, ids = s["case"], s["x"], s["indices"].long()
    T, E, K = case["tokens"], case["experts"], case["topk"]
    if T * K <= E:                       # the chosen experts' weights, one copy for each choice
        which, rows = ids.clamp(min=0).flatten(), x.float().repeat_interleave(K, 0)[:, None]
        up, down = s["up"][which], s["down"][which]
    else:                                # every expert on every token
        which, rows = slice(None), x.float().expand(E, T, -1)
        up, down = s["up"], s["down"]
    h = torch.bmm(rows, up.float().transpose(1, 2))
    if s["up_bias"] is not None:
        h = h + s["up_bias"][which].float()[:, None]
    h = activation(h, case["act"], case["inner"])
    y = torch.bmm(h, down.float().transpose(1, 2))
    if s["down_bias"] is not None:
        y = y + s["down_bias"][which].float()[:, None]
    if T * K <= E:
        y = y.view(T, K, -1)
    else:
        y = y[ids.clamp(min=0), torch.arange(T, device=x.device)[:, None]]
    out = (y * torch.where(ids >= 0, s["weights"], torch.zeros_like(s["weights"]))[..., None]).sum(1)
    return (out + s["residual"].float() if s["residual"] is not None else out).to(x.dtype)


PLAIN = {"norm": plain_norm, "norm_backward": plain_norm_backward, "save": plain_save, "restore": plain_restore,
         "grad": plain_grad, "few": plain_few}


# ------------------------------------------------------ one pass, and its cost

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return PLAIN[op](s)
    import combine_ep_layout_06_gb300 as ep
    if op == "norm":
        out = ep.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, quantize=case["eight"])
        return out if isinstance(out, tuple) else (out,)
    if op == "norm_backward":
        return ep.rms_norm_backward(s["grad"], s["x"], s["weight"], grad_total=s["grad_total"], eps=EPS)
    if op == "save":
        return ep.checkpoint(s["pre"], s["count"], s["offset"])
    if op == "restore":
        return ep.checkpoint_restore(s["codes"], s["scales"], s["count"], s["offset"], activation=case["act"],
                                     dtype=DTYPES[case["dtype"]])
    if op == "grad":
        dx, dw, _ = ep.expert_product_backward(s["grad"], s["x"], s["weight"], s["count"], s["offset"], pre=s["codes"],
                                               pre_scales=s["scales"], activation=case["act"])
        return dx, dw
    return ep.moe_few_tokens(s["x"], s["weights"], s["indices"], s["up"], s["down"], activation=case["act"],
                             up_bias=s["up_bias"], down_bias=s["down_bias"], residual=s["residual"])


def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op.startswith("norm"):
        values, H = case["rows"] * case["width"], case["width"]
        if op == "norm":
            result = values + values // BLOCK * 4 if case["eight"] else values * size
            return {"bytes": values * size * (3 if case["residual"] else 1) + result + H * size, "flops": 5.0 * values}
        return {"bytes": values * size * (4 if case["total"] else 3) + 2 * H * size, "flops": 10.0 * values}
    if op == "few":
        ids = [e for row in choices(case) for e in row if e >= 0]
        T, H, F, used, pairs = case["tokens"], case["hidden"], case["inner"], len(set(ids)), len(ids)
        moved = used * H * (wide(case) + F) + T * H * (3 if case["residual"] else 2)
        moved += used * (wide(case) + H) if case["bias"] else 0
        return {"bytes": moved * size + T * case["topk"] * 8, "flops": 2.0 * pairs * H * (wide(case) + F)}
    rows, n = case["rows"], case["n"]
    kept = rows * (wide(case) + -(-wide(case) // BLOCK) * 4)
    if op == "save":
        return {"bytes": rows * wide(case) * size + kept, "flops": 3.0 * rows * wide(case)}
    if op == "restore":
        return {"bytes": kept + rows * n * size, "flops": 6.0 * rows * wide(case)}
    k, used = case["k"], sum(c > 0 for c in group_counts(case))
    moved = (used + case["groups"]) * wide(case) * k + rows * (2 * k + n)
    return {"bytes": size * moved + kept, "flops": 4.0 * rows * wide(case) * k}


# ------------------------------------------------------- 64-bit definitions

def exact_codes(v):
    """Scales, and the codes before they are rounded."""
    scales = torch.stack([b.abs().amax(-1) for b in v.split(BLOCK, -1)], -1) / 448.0
    return torch.cat([b / scales[..., i:i + 1].clamp(min=1e-300) for i, b in enumerate(v.split(BLOCK, -1))], -1), scales


def exact_activation(name):
    f = torch.nn.functional
    return {"relu": torch.relu, "gelu": f.gelu, "silu": f.silu,
            "swiglu": lambda v: f.silu(v.chunk(2, -1)[0]) * v.chunk(2, -1)[1]}[name]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        total = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
        h = total.double()                  # the norm is of the rounded sum
        y = h / torch.sqrt(h.pow(2).sum(-1, keepdim=True) / case["width"] + EPS) * s["weight"].double()
        whole = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        return (exact_codes(y) if case["eight"] else (y,)) + ((whole,) if s["residual"] is not None else ())
    if op == "norm_backward":
        h, w = s["x"].double().requires_grad_(True), s["weight"].double().requires_grad_(True)
        goal = (h / torch.sqrt(h.pow(2).sum(-1, keepdim=True) / case["width"] + EPS) * w * s["grad"].double()).sum()
        if s["grad_total"] is not None:
            goal = goal + (h * s["grad_total"].double()).sum()
        return torch.autograd.grad(goal, (h, w))
    if op == "save":
        return exact_codes(s["pre"].double())
    act = exact_activation(case["act"])
    if op == "few":
        T, H = s["x"].shape
        out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        ids = choices(case)
        for e in sorted({e for row in ids for e in row if e >= 0}):
            where = [(t, row.index(e)) for t, row in enumerate(ids) if e in row]
            t, j = (torch.tensor(v, device="cuda") for v in zip(*where))
            h = s["x"][t].double() @ s["up"][e].double().T
            h = act(h if s["up_bias"] is None else h + s["up_bias"][e].double())
            y = h @ s["down"][e].double().T
            y = y if s["down_bias"] is None else y + s["down_bias"][e].double()
            out[t] += y * s["weights"][t, j].double()[:, None]
        return out if s["residual"] is None else out + s["residual"].double()
    n_blocks = s["scales"].shape[-1]
    v = s["codes"].double()
    v = torch.cat([v[..., i * BLOCK:(i + 1) * BLOCK] * s["scales"][..., i:i + 1].double() for i in range(n_blocks)], -1)
    if op == "restore":
        return act(v)
    v.requires_grad_(True)
    d, = torch.autograd.grad(act(v), v, s["grad"].double())
    G, per, counts = case["groups"], case["groups"] // case["ranks"], group_counts(case)
    dx, dw = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda"), torch.zeros(s["weight"].shape, dtype=torch.float64, device="cuda")
    start = 0
    for g in range(G):
        start = 0 if g % per == 0 else start
        at = (g // per, slice(start, start + counts[g]))
        start += counts[g]
        dx[at], dw[g] = d[at] @ s["weight"][g].double(), d[at].T @ s["x"][at].double()
    return dx, dw
