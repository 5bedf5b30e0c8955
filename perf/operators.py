"""The operators around the expert-parallel token path, and the cases they are measured on.

Three operators, each with its gradient:

route           top-k routing: expert ids and weights of every token from its router logits
balance_loss    the loss that evens out the experts' loads, with per-expert counts, and the log-sum-exp (z) loss
expert_product  one matrix product per expert over rows grouped by expert, with bias, activation and residual

``own`` chooses between the plain forms below and the package's kernels.  A group is an expert (of a
rank, where rows come in one segment per rank); its rows are offset[g] .. offset[g] + count[g] - 1.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FLT_MAX = torch.finfo(torch.float32).max
SQRT2 = math.sqrt(2.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One decoded token's logits over 256 experts: what a single-stream server calls once per layer.
        dict(name="route_one_token", op="route", ranks=1, tokens=1, experts=256, topk=8, dtype="bf16", score="sigmoid",
             renormalize=True, scale=2.5, bias=True, masked=False, ragged=False),
        # A training or prefill batch of 8 ranks x 4096 tokens over 256 experts.
        dict(name="route_batch", op="route", ranks=8, tokens=4096, experts=256, topk=8, dtype="bf16", score="softmax",
             renormalize=True, scale=1.0, bias=True, masked=False, ragged=True),
        # Few experts, many tokens: 8 ranks x 16384 tokens, top-2 of 8, two experts closed by a mask.
        dict(name="route_few_experts", op="route", ranks=8, tokens=16384, experts=8, topk=2, dtype="fp32", score="softmax",
             renormalize=False, scale=1.0, bias=False, masked=True, ragged=False),
        # The router's whole gradient in training: of the weights and of the balance loss, in one call.
        dict(name="route_grad_batch", op="route_backward", ranks=8, tokens=4096, experts=256, topk=8, dtype="fp32",
             score="softmax", renormalize=True, scale=1.0, bias=False, masked=False, ragged=True, loss=True),
        # The balance loss of a small batch with an odd number of experts.
        dict(name="balance_small", op="balance", ranks=2, tokens=128, experts=77, topk=3, dtype="fp16", masked=True, ragged=True,
             z=True),
        # The balance loss of a training batch.
        dict(name="balance_batch", op="balance", ranks=8, tokens=4096, experts=256, topk=8, dtype="bf16", masked=False,
             ragged=False, z=True),
        # Its gradient.
        dict(name="balance_grad_batch", op="balance_backward", ranks=8, tokens=4096, experts=256, topk=8, dtype="bf16",
             masked=False, ragged=False, z=True),
        # A small model's experts at decode: latency.
        dict(name="product_tiny", op="product", ranks=2, groups=8, rows=16, k=256, n=512, dtype="bf16", act="silu",
             bias=True, residual=False, pre=False, empty=0, layout=3),
        # One rank's 32 experts at decode, 128 routed rows: every expert's gate and up weights are read for a few rows each.
        dict(name="product_decode", op="product", ranks=1, groups=32, rows=128, k=7168, n=1792, dtype="bf16", act="swiglu",
             bias=False, residual=False, pre=False, empty=2, layout=5),
        # Prefill of the same experts, gate and up with the gated activation, pre-activations kept as training keeps them.
        dict(name="product_prompt", op="product", ranks=1, groups=32, rows=32768, k=7168, n=1792, dtype="bf16", act="swiglu",
             bias=False, residual=False, pre=True, empty=0, layout=7),
        # Down projection over 8 ranks with one expert each, two ranks' experts idle, odd row counts, bias and residual.
        dict(name="product_down", op="product", ranks=1, groups=8, rows=32761, k=3584, n=4096, dtype="fp16", act="none",
             bias=True, residual=True, pre=False, empty=2, layout=11),
        # The gradient of gate and up: inputs, weights and biases of 8 experts.
        dict(name="product_grad", op="product_backward", ranks=2, groups=8, rows=16384, k=4096, n=1792, dtype="bf16",
             act="swiglu", bias=True, empty=1, layout=13),
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "balance", "balance_backward", "product", "product", "product", "product_backward"])
    if not op.startswith("product"):
        experts = spread(rng, 8, 256)
        case = dict(op=op, ranks=rng.choice([1, 2, 8]), tokens=spread(rng, 1, 4096), experts=experts,
                    topk=rng.randint(1, min(8, experts)), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    masked=rng.random() < 0.3, ragged=rng.random() < 0.5)
        if op.startswith("route"):
            case.update(score=rng.choice(["softmax", "sigmoid"]), renormalize=rng.random() < 0.5,
                        scale=rng.choice([1.0, 2.5]), bias=op == "route" and rng.random() < 0.5)
        if op == "route_backward":
            case["loss"] = rng.random() < 0.5
        if op.startswith("balance"):
            case["z"] = rng.random() < 0.5
        return case
    ranks = rng.choice([1, 1, 2])
    groups = ranks * spread(rng, 1, 32 // ranks)
    sizes = [8 * spread(rng, 8, 512) for _ in range(2)]
    sizes = [s + 8 if s == 3072 else s for s in sizes]
    rows = ranks * max(1, spread(rng, 1, 16384) // ranks)
    case = dict(op=op, ranks=ranks, groups=groups, rows=rows, k=sizes[0], n=sizes[1], dtype=rng.choice(["bf16", "fp16"]),
                act=rng.choice(["none", "relu", "gelu", "silu", "swiglu"]), bias=rng.random() < 0.5,
                empty=rng.randint(0, (groups // ranks - 1) // 4), layout=rng.randrange(1 << 20))
    if op == "product":
        case.update(residual=rng.random() < 0.4, pre=rng.random() < 0.4)
    # below the largest listed cases, in memory and in work
    while case["groups"] > ranks and case["groups"] * case["k"] * case["n"] > 1 << 27:
        case["groups"] -= ranks
    case["empty"] = min(case["empty"], (case["groups"] // ranks - 1) // 4)
    while work(case)["flops"] > 6e11:
        case["rows"] = ranks * max(1, case["rows"] // ranks // 2)
    return case


def group_counts(case):
    """Rows of every group, from the case alone: uneven, `empty` groups of each rank without any."""
    rng = random.Random(case["layout"])
    per = case["groups"] // case["ranks"]
    counts = []
    for _ in range(case["ranks"]):
        share = [rng.uniform(0.6, 1.4) for _ in range(per)]
        for g in rng.sample(range(per), min(case["empty"], per - 1)):
            share[g] = 0.0
        rows = case["rows"] // case["ranks"]
        ends, run, total = [], 0.0, sum(share)
        for s in share:
            run += s
            ends.append(int(round(rows * run / total)))
        ends[-1] = rows
        counts += [b - a for a, b in zip([0] + ends[:-1], ends)]
    return counts


def token_counts(case):
    """Tokens present on every rank: full, or ragged with one rank empty."""
    ranks, tokens = case["ranks"], case["tokens"]
    if not case["ragged"]:
        return [tokens] * ranks
    rng = random.Random(tokens * 131 + ranks)
    counts = [rng.randint((tokens + 1) // 2, tokens) for _ in range(ranks)]
    if ranks > 2:
        counts[rng.randrange(1, ranks)] = 0
    return counts


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    s = dict(case=case)
    if case["op"].startswith("product"):
        dtype, act = DTYPES[case["dtype"]], case["act"]
        R, G, k, n = case["ranks"], case["groups"], case["k"], case["n"]
        wide = 2 * n if act == "swiglu" else n
        cap = case["rows"] // R
        counts = group_counts(case)
        per = G // R
        offsets = [sum(counts[g - g % per:g]) for g in range(G)]
        s["count"] = torch.tensor(counts, dtype=torch.int32, device="cuda").view(R, per)
        s["offset"] = torch.tensor(offsets, dtype=torch.int32, device="cuda").view(R, per)
        # the plain form's padded layout: row i of group g stands at g * most + i
        most = max(counts)
        first = torch.tensor([g // per * cap + o for g, o in enumerate(offsets)], device="cuda")
        step = torch.arange(most, device="cuda")
        s["slots"] = (first[:, None] + step).clamp(max=R * cap - 1)
        s["here"] = step < torch.tensor(counts, device="cuda")[:, None]
        s["x"] = normal(R, cap, k, dtype=dtype)
        s["weight"] = torch.empty(G, wide, k, dtype=dtype, device="cuda")
        for g in range(G):
            s["weight"][g] = normal(wide, k, std=k ** -0.5, dtype=dtype)
        s["bias"] = normal(G, wide, std=0.1, dtype=dtype) if case["bias"] else None
        if case["op"] == "product":
            s["residual"] = normal(R, cap, n, dtype=dtype) if case["residual"] else None
        else:
            s["pre"] = normal(R, cap, wide, dtype=dtype)
            s["grad"] = normal(R, cap, n, std=0.1, dtype=dtype)
        return s
    R, T, E, K = case["ranks"], case["tokens"], case["experts"], case["topk"]
    logits = normal(R, T, E, std=1.5)
    if case["masked"]:      # some experts are closed, and some tokens see none at all
        closed = torch.rand((R, T, E), generator=gen, device="cuda") < 0.2
        closed |= torch.rand((R, T, 1), generator=gen, device="cuda") < 0.01
        logits.masked_fill_(closed, -math.inf)
    s["logits"] = logits.to(DTYPES[case["dtype"]])
    s["num_tokens"] = token_counts(case)
    s["bias"] = normal(E, std=0.1) if case.get("bias") else None
    if case["op"] != "route":
        s["indices"] = torch.argsort(torch.rand((R, T, E), generator=gen, device="cuda"), dim=-1)[..., :K].to(torch.int32).contiguous()
        s["grad_weights"] = normal(R, T, K)
        s["grad_loss"] = torch.rand((), generator=gen, device="cuda") + 0.5
        present = torch.arange(T, device="cuda") < torch.tensor(s["num_tokens"], device="cuda")[:, None]
        s["counts"] = torch.bincount(s["indices"][present].flatten().long(), minlength=E).to(torch.int32)
    return s


# ------------------------------------------------------------ plain forms

def present_rows(s, like):
    T = s["case"]["tokens"]
    n = torch.tensor(s["num_tokens"], device=like.device)
    return (torch.arange(T, device=like.device) < n[:, None])[..., None]


def finite_logits(s):
    """32-bit logits with what is not a number as -inf, +inf as the largest number, and the rows that are present."""
    x = s["logits"].float()
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x).clamp(max=FLT_MAX)
    return x, present_rows(s, x)


def probabilities(x):
    """softmax over the last axis (a row of -inf gives zeros), and its log-sum-exp."""
    top = x.amax(-1, keepdim=True)
    open_ = top > -math.inf
    e = torch.exp(x - torch.where(open_, top, torch.zeros_like(top)))
    total = e.sum(-1, keepdim=True)
    p = torch.where(open_, e / torch.where(open_, total, torch.ones_like(total)), torch.zeros_like(e))
    return p, torch.where(open_, top + torch.log(total), torch.zeros_like(total))


def scores(x, score):
    return probabilities(x)[0] if score == "softmax" else 1.0 / (1.0 + torch.exp(-x))


def chosen_scores(case, x, ids):
    """The chosen experts' scores: those that a renormalised softmax needs are taken over the chosen alone."""
    if case["score"] == "softmax" and case["renormalize"]:
        return probabilities(torch.gather(x, -1, ids))[0]
    return torch.gather(scores(x, case["score"]), -1, ids)


def plain_route(s):
    case = s["case"]
    x, present = finite_logits(s)
    key = x if s["bias"] is None else x + s["bias"]
    ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :case["topk"]]
    w = chosen_scores(case, x, ids)
    if case["renormalize"] and case["score"] == "sigmoid":
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / torch.where(total > 0, total, torch.ones_like(total)), torch.zeros_like(w))
    w = torch.where(present, w * case["scale"], torch.zeros_like(w))
    return w, torch.where(present, ids, torch.full_like(ids, -1)).to(torch.int32)


def balance_slope(s, p, lse, present, topk, balance_coef, z_coef):
    """The gradient of the balance and z losses by the logits, times the loss's own gradient."""
    n = sum(s["num_tokens"])
    f = s["counts"].float() * (s["case"]["experts"] / (topk * max(1, n)))
    inner = (p * f).sum(-1, keepdim=True)
    d = p * (balance_coef * (f - inner) + 2.0 * z_coef * lse) * (s["grad_loss"] / max(1, n))
    return torch.where(present, d, torch.zeros_like(d))


def plain_route_backward(s):
    case = s["case"]
    x, present = finite_logits(s)
    ids = s["indices"].long()
    g = torch.where(present, s["grad_weights"] * case["scale"], torch.zeros_like(s["grad_weights"]))
    v = chosen_scores(case, x, ids)
    if case["score"] == "softmax":
        inner = (g * v).sum(-1, keepdim=True)
        d = torch.zeros_like(x)
        if case["renormalize"]:
            d.scatter_(-1, ids, v * (g - inner))
        else:
            d.scatter_(-1, ids, v * g)
            d -= scores(x, "softmax") * inner
    else:
        dv = g
        if case["renormalize"]:
            total = v.sum(-1, keepdim=True)
            some = total > 0
            total = torch.where(some, total, torch.ones_like(total))
            dv = torch.where(some, (g - (g * v).sum(-1, keepdim=True) / total) / total, torch.zeros_like(g))
        d = torch.zeros_like(x).scatter_(-1, ids, dv * v * (1.0 - v))
    if case["loss"]:
        p, lse = probabilities(x)
        d = d + balance_slope(s, p, lse, present, case["topk"], *coefs(case))
    return torch.where(present, d, torch.zeros_like(d)).to(s["logits"].dtype)


def coefs(case):
    return 0.01, 0.001 if case.get("z", True) else 0.0


def plain_balance(s):
    case = s["case"]
    balance_coef, z_coef = coefs(case)
    E, n = case["experts"], sum(s["num_tokens"])
    x, present = finite_logits(s)
    p, lse = probabilities(x)
    ids = torch.where(present, s["indices"].long(), torch.full_like(s["indices"].long(), E)).reshape(-1)
    counts = torch.zeros(E + 1, dtype=torch.int32, device=x.device).index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))[:E]
    mean = torch.where(present, p, torch.zeros_like(p)).sum((0, 1)) / max(1, n)
    balance = (counts.float() * (E / (case["topk"] * max(1, n))) * mean).sum()
    z = torch.where(present, lse * lse, torch.zeros_like(lse)).sum() / max(1, n)
    return torch.stack([balance_coef * balance + z_coef * z, balance, z]), counts, mean


def plain_balance_backward(s):
    x, present = finite_logits(s)
    p, lse = probabilities(x)
    return balance_slope(s, p, lse, present, s["case"]["topk"], *coefs(s["case"])).to(s["logits"].dtype)


def activation(v, act, n):
    if act == "relu":
        return v.clamp(min=0)
    if act == "gelu":
        return v * 0.5 * (1.0 + torch.erf(v / SQRT2))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "swiglu":
        return v[..., :n] / (1.0 + torch.exp(-v[..., :n])) * v[..., n:]
    return v


def padded(s, t):
    """[R][cap][c] rows as [G][most][c] in 32 bits, zeros where a group has no such row."""
    t = t.reshape(-1, t.shape[-1])[s["slots"]].float()
    return torch.where(s["here"][..., None], t, torch.zeros_like(t))


def compact(s, t, shape, dtype):
    """[G][most][c] back to the rows in place, rounded to their type."""
    out = torch.zeros((shape[0] * shape[1], t.shape[-1]), dtype=dtype, device=t.device)
    out[s["slots"][s["here"]]] = t[s["here"]].to(dtype)
    return out.view(shape[0], shape[1], -1)


def plain_product(s):
    case, x = s["case"], s["x"]
    pre = torch.bmm(padded(s, x), s["weight"].float().transpose(1, 2))
    if s["bias"] is not None:
        pre = pre + s["bias"].float()[:, None]
    y = activation(pre, case["act"], case["n"])
    if s["residual"] is not None:
        y = y + padded(s, s["residual"])
    y = compact(s, y, x.shape, x.dtype)
    return (y, compact(s, pre, x.shape, x.dtype)) if case["pre"] else y


def plain_product_backward(s):
    case, x, n = s["case"], s["x"], s["case"]["n"]
    g, v = padded(s, s["grad"]), padded(s, s["pre"])
    act = case["act"]
    if act == "relu":
        d = torch.where(v > 0, g, torch.zeros_like(g))
    elif act == "gelu":
        d = g * (0.5 * (1.0 + torch.erf(v / SQRT2)) + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi))
    elif act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-v))
        d = g * sig * (1.0 + v * (1.0 - sig))
    elif act == "swiglu":
        gate, up = v[..., :n], v[..., n:]
        sig = 1.0 / (1.0 + torch.exp(-gate))
        d = torch.cat([g * up * sig * (1.0 + gate * (1.0 - sig)), g * gate * sig], -1)
    else:
        d = g
    dx = compact(s, torch.bmm(d, s["weight"].float()), x.shape, x.dtype)
    dw = torch.bmm(d.transpose(1, 2), padded(s, x)).to(x.dtype)
    return (dx, dw, d.sum(1).to(x.dtype)) if case["bias"] else (dx, dw)


PLAIN = {"route": plain_route, "route_backward": plain_route_backward, "balance": plain_balance,
         "balance_backward": plain_balance_backward, "product": plain_product, "product_backward": plain_product_backward}


# ------------------------------------------------------ one pass, and its cost

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return PLAIN[op](s)
    import combine_ep_layout_06_gb300 as ep
    if op == "route":
        return ep.route(s["logits"], case["topk"], score=case["score"], renormalize=case["renormalize"], scale=case["scale"],
                        bias=s["bias"], num_tokens=s["num_tokens"])
    if op == "route_backward":
        balance_coef, z_coef = coefs(case)
        loss = dict(grad_loss=s["grad_loss"], counts=s["counts"], balance_coef=balance_coef, z_coef=z_coef) if case["loss"] else {}
        return ep.route_backward(s["grad_weights"], s["logits"], s["indices"], score=case["score"],
                                 renormalize=case["renormalize"], scale=case["scale"], num_tokens=s["num_tokens"], **loss)
    if op == "balance":
        balance_coef, z_coef = coefs(case)
        return ep.balance_loss(s["logits"], s["indices"], balance_coef=balance_coef, z_coef=z_coef, num_tokens=s["num_tokens"])
    if op == "balance_backward":
        balance_coef, z_coef = coefs(case)
        return ep.balance_loss_backward(s["grad_loss"], s["logits"], s["counts"], case["topk"], balance_coef=balance_coef,
                                        z_coef=z_coef, num_tokens=s["num_tokens"])
    if op == "product":
        return ep.expert_product(s["x"], s["weight"], s["count"], s["offset"], bias=s["bias"], activation=case["act"],
                                 residual=s["residual"], save_pre=case["pre"])
    dx, dw, db = ep.expert_product_backward(s["grad"], s["x"], s["weight"], s["count"], s["offset"], pre=s["pre"],
                                            activation=case["act"], bias_grad=case["bias"])
    return (dx, dw, db) if case["bias"] else (dx, dw)


def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op.startswith("product"):
        counts = group_counts(case)
        used = sum(c > 0 for c in counts)
        rows, k, n = sum(counts), case["k"], case["n"]
        wide = 2 * n if case["act"] == "swiglu" else n
        weights = used * wide * k
        if op == "product":
            moved = weights + rows * (k + n) + (used * wide if case["bias"] else 0)
            moved += (rows * n if case["residual"] else 0) + (rows * wide if case["pre"] else 0)
            return {"bytes": size * moved, "flops": 2.0 * rows * wide * k}
        everything = case["groups"] * wide * (k + (1 if case["bias"] else 0))
        saved = wide if case["act"] != "none" else 0
        return {"bytes": size * (weights + everything + rows * (k + n + saved + k)), "flops": 4.0 * rows * wide * k}
    rows, all_rows = sum(token_counts(case)), case["ranks"] * case["tokens"]
    E, K = case["experts"], case["topk"]
    if op == "route":
        return {"bytes": rows * E * size + all_rows * K * 8 + (E * 4 if case["bias"] else 0), "flops": rows * E * 4.0}
    if op == "route_backward":
        sparse = not case["loss"] and (case["renormalize"] or case["score"] == "sigmoid")
        read = rows * (K * 32 if sparse else E * size)      # the chosen logits alone: one 32-byte sector each
        read = min(read, rows * E * size)
        return {"bytes": read + rows * K * 8 + all_rows * E * size + (E * 4 if case["loss"] else 0), "flops": rows * E * 8.0}
    if op == "balance":
        return {"bytes": rows * (E * size + K * 4) + E * 8 + 12, "flops": rows * E * 6.0}
    return {"bytes": rows * E * size + all_rows * E * size + E * 4, "flops": rows * E * 10.0}


# ------------------------------------------------------- 64-bit definitions

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("product"):
        return exact_product(s)
    E, K = case["experts"], case["topk"]
    logits = torch.nan_to_num(s["logits"].double(), nan=-math.inf, posinf=float(FLT_MAX), neginf=-math.inf)
    logits.requires_grad_(True)
    keep = torch.zeros(logits.shape[:2], dtype=torch.bool, device=logits.device)
    for r, t in enumerate(s["num_tokens"]):
        keep[r, :t] = True
    some = keep & (logits.detach() > -math.inf).any(-1)
    rows = logits[some]                                  # the tokens that are there and see an expert
    n = max(1, sum(s["num_tokens"]))

    def weights(ids):
        picked = rows.gather(1, ids)
        if case["score"] == "sigmoid":
            v = torch.sigmoid(picked)
            if case["renormalize"]:
                total = v.sum(1, keepdim=True)
                v = v / torch.where(total > 0, total, torch.ones_like(total))
            return v * case["scale"]
        if not case["renormalize"]:
            return torch.exp(picked - torch.logsumexp(rows, 1, keepdim=True)) * case["scale"]
        shut = torch.isinf(picked).all(1, keepdim=True)  # every chosen expert is closed
        v = torch.softmax(torch.where(shut, torch.zeros_like(picked), picked), 1)
        return torch.where(shut, torch.zeros_like(v), v) * case["scale"]

    if case["op"] == "route":
        key = s["logits"].float() if s["bias"] is None else s["logits"].float() + s["bias"]
        ids = torch.sort(key[some], dim=1, descending=True, stable=True).indices[:, :K]
        out = torch.zeros(logits.shape[:2] + (K,), dtype=torch.float64, device=logits.device)
        out[some] = weights(ids).detach()
        return out, None
    if case["op"] == "balance":
        f = torch.bincount(s["indices"][keep].flatten().long(), minlength=E).double() * E / (K * n)
    else:
        f = s["counts"].double() * E / (K * n)
    share = torch.softmax(rows, 1).sum(0) / n
    balance, z = (f * share).sum(), torch.logsumexp(rows, 1).square().sum() / n
    balance_coef, z_coef = coefs(case)
    loss = balance_coef * balance + z_coef * z
    if case["op"] == "balance":
        return torch.stack([loss, balance, z]).detach(), None, share.detach()
    goal = loss * s["grad_loss"].double() if case["op"] == "balance_backward" or case["loss"] else 0.0
    if case["op"] == "route_backward":
        goal = goal + (weights(s["indices"][some].long()) * s["grad_weights"][some].double()).sum()
    grad, = torch.autograd.grad(goal, logits)
    return torch.nan_to_num(grad, nan=0.0)               # 0 * inf at closed experts


def exact_product(s):
    case, x = s["case"], s["x"]
    R, G, n = case["ranks"], case["groups"], case["n"]
    per, counts = G // R, group_counts(case)
    wide = s["weight"].shape[1]

    def act(v):
        name = case["act"]
        if name == "swiglu":
            return torch.nn.functional.silu(v[:, :n]) * v[:, n:]
        return {"none": lambda t: t, "relu": torch.relu, "silu": torch.nn.functional.silu,
                "gelu": torch.nn.functional.gelu}[name](v)

    f64 = dict(dtype=torch.float64, device=x.device)
    if case["op"] == "product":
        y, pre = torch.zeros(x.shape[:2] + (n,), **f64), torch.zeros(x.shape[:2] + (wide,), **f64)
    else:
        dx, dw, db = torch.zeros(x.shape, **f64), torch.zeros(s["weight"].shape, **f64), torch.zeros((G, wide), **f64)
    start = 0
    for g in range(G):
        start = 0 if g % per == 0 else start
        rows = (g // per, slice(start, start + counts[g]))
        start += counts[g]
        w, xs = s["weight"][g].double(), x[rows].double()
        if case["op"] == "product":
            v = xs @ w.T
            if s["bias"] is not None:
                v += s["bias"][g].double()
            pre[rows] = v
            y[rows] = act(v) + (s["residual"][rows].double() if s["residual"] is not None else 0.0)
        else:
            v = s["pre"][rows].double().requires_grad_(True)
            d, = torch.autograd.grad(act(v), v, s["grad"][rows].double())
            dx[rows], dw[g], db[g] = d @ w, d.T @ xs, d.sum(0)
    if case["op"] == "product":
        return (y, pre) if case["pre"] else y
    return (dx, dw, db) if case["bias"] else (dx, dw)
