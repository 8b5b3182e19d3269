"""The library's softmax-over-codes operators as cases to be measured.

Five operators: scores of given tokens from logits and their gradient, the same two fused with the
product that makes the logits, and a mixture-of-experts layer for a few tokens. ``run`` makes
the calls of ``gmm_em_amd.ops`` where ``own`` is true and computes the same in plain torch operations in 32
bits where it is not; ``exact`` computes it in 64 bits from the definitions.

Inputs whose order decides an output (the alternatives of a head, the experts of a router) lie on an
8-bit grid, as quantised descriptors and codebooks do (the library's headline rows are integers): every sum of
products is then exact in 32 bits, so that each right implementation ranks them alike, ties included.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # one decoding step's logits of a 16384-code vocabulary: latency
        {"name": "score_one_row", "op": "score", "n": 1, "v": 16384, "m": 4, "dtype": "f32", "masked": False},
        # a prompt's logits with a grammar mask: odd sizes, some rows with no code left
        {"name": "score_masked_odd", "op": "score", "n": 333, "v": 40009, "m": 16, "dtype": "f32", "masked": True},
        # a batch of sequences scored at once
        {"name": "score_batch", "op": "score", "n": 4096, "v": 32768, "m": 4, "dtype": "bf16", "masked": False},
        # gradient of a small ragged batch, some codes masked
        {"name": "score_grad_odd", "op": "score_grad", "n": 257, "v": 10007, "dtype": "f32", "masked": True},
        # gradient of a training batch
        {"name": "score_grad_batch", "op": "score_grad", "n": 4096, "v": 32768, "dtype": "bf16", "masked": False},
        # a decoding step of four sequences on the wide workload's sizes (768 dims, 16384 codes)
        {"name": "head_decode", "op": "head", "n": 4, "d": 768, "v": 16384, "m": 4, "dtype": "bf16"},
        # integer descriptors against 1024 codes, two lists a row (96 dims, as the descriptor workload)
        {"name": "head_descriptor", "op": "head", "n": 5003, "d": 96, "v": 1024, "m": 2, "dtype": "f32"},
        # the loss of a training batch on the wide workload's sizes
        {"name": "head_batch", "op": "head", "n": 8192, "d": 768, "v": 16384, "m": 0, "dtype": "bf16"},
        # gradient of a small head in 32 bits, odd in every direction
        {"name": "head_grad_odd", "op": "head_grad", "n": 777, "d": 100, "v": 1001, "dtype": "f32"},
        # gradient of the training batch
        {"name": "head_grad_batch", "op": "head_grad", "n": 8192, "d": 768, "v": 16384, "dtype": "bf16"},
        # one token through two of 64 experts: latency
        {"name": "moe_one_token", "op": "moe", "n": 1, "d": 768, "f": 2048, "e": 64, "m": 2, "dtype": "bf16"},
        # a decoding batch that reaches nearly every expert
        {"name": "moe_batch", "op": "moe", "n": 64, "d": 2048, "f": 1408, "e": 64, "m": 4, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["score", "score_grad", "head", "head_grad", "moe"])
    c = {"op": op, "dtype": rng.choice(["f32", "bf16"])}
    wide = 2 if c["dtype"] == "f32" else 1
    if op in ("score", "score_grad"):
        c["n"], c["v"] = _log(rng, 1, 8192), _log(rng, 100, 65536)
        c["n"] = max(1, min(c["n"], 4096 * 32768 // (wide * c["v"])))
        c["masked"] = rng.random() < 0.5
        if op == "score":
            c["m"] = rng.randint(0, 16)
    elif op in ("head", "head_grad"):
        c["n"], c["v"], c["d"] = _log(rng, 1, 8192), _log(rng, 100, 32768), _log(rng, 32, 1024)
        # 32-bit products cost several 16-bit ones
        c["n"] = max(1, min(c["n"], 8192 * 768 * 16384 // (6 * (wide - 1) + 1) // (c["v"] * c["d"])))
        if op == "head":
            c["m"] = rng.choice([0, 0, rng.randint(1, 16)])
    else:
        c["n"], c["e"], c["m"] = _log(rng, 1, 64), _log(rng, 8, 128), rng.randint(1, 4)
        c["d"], c["f"] = _log(rng, 96, 2048), _log(rng, 128, 4096)
        # an expert, and a token's pass through its experts, cost at most the listed batch's
        c["f"] = max(8, min(c["f"], 64 * 2048 * 1408 // (wide * c["e"] * c["d"])))
    return c


def _experts_hit(c):
    """Experts that at least one of the tokens picks, for even picks."""
    return c["e"] * (1.0 - (1.0 - c["m"] / c["e"]) ** c["n"])


def work(case):
    c, es = case, SIZE[case["dtype"]]
    n = c["n"]
    if c["op"] == "score":
        return {"bytes": n * c["v"] * es + n * (20 + 8 * c["m"]), "flops": 5.0 * n * c["v"]}
    if c["op"] == "score_grad":
        return {"bytes": 2 * n * c["v"] * es + n * 24, "flops": 8.0 * n * c["v"]}
    if c["op"] == "head":
        return {"bytes": (n + c["v"]) * c["d"] * es + n * (20 + 8 * c["m"]),
                "flops": 2.0 * n * c["v"] * c["d"]}
    if c["op"] == "head_grad":
        return {"bytes": 2 * (n + c["v"]) * c["d"] * es + n * 24, "flops": 6.0 * n * c["v"] * c["d"]}
    return {"bytes": _experts_hit(c) * 3 * c["f"] * c["d"] * es + (c["e"] + 2 * n) * c["d"] * es
            + 8 * n * c["m"],
            "flops": 6.0 * n * c["m"] * c["f"] * c["d"] + 2.0 * n * c["e"] * c["d"]}


def _grid(t, step, most):
    """Values on a grid of `step` with at most 8 bits."""
    return (t / step).round_().clamp_(-most, most) * step


def _norm(logits):
    """The row's largest logit and the log of the sum of exp(l - largest); 0 where nothing is left."""
    top = logits.max(1, keepdim=True).values
    none = top == -math.inf
    rest = torch.exp(logits - top.masked_fill(none, 0.0)).sum(1, keepdim=True).log()
    return torch.cat([top, rest.masked_fill(none, 0.0)], 1)


def prepare(case, seed):
    c, dt = case, TYPES[case["dtype"]]
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    s = {"case": dict(c)}
    n = c["n"]
    if c["op"] == "moe":
        d, f, e = c["d"], c["f"], c["e"]
        s["x"] = _grid(normal(n, d), 2.0 ** -5, 127).to(dt)
        s["gate"] = _grid(normal(e, d) / math.sqrt(d), 2.0 ** -10, 127).to(dt)
        s["w_in"] = (normal(e, 2 * f, d) / math.sqrt(d)).to(dt)
        s["w_out"] = (normal(e, d, f) / math.sqrt(f)).to(dt)
        return s
    v = c["v"]
    # codes are met with uneven frequency; some places carry none
    s["targets"] = (v * uniform(n) ** 2).to(torch.int32).clamp_(max=v - 1)
    s["targets"][uniform(n) < 0.05] = -1
    s["scale"] = 1.25  # a temperature of 0.8
    if c["op"] in ("score", "score_grad"):
        x = 2.5 * normal(n, v)
        if c["masked"]:
            x[uniform(n, v) < 0.3] = -math.inf
            low = uniform(n) < 0.2  # rows masked with the type's lowest value instead
            x[low] = x[low].clamp_(min=torch.finfo(dt).min)
            x[uniform(n) < 0.05] = -math.inf  # rows with nothing left
        s["logits"] = x.to(dt)
    elif c["op"] == "head" and c["m"] > 0:
        d = c["d"]
        s["hidden"] = _grid(normal(n, d), 2.0 ** -5, 127).to(dt)
        s["weight"] = _grid(normal(v, d), 2.0 ** -5, 127).mul_(2.0 ** -3).to(dt)
        s["scale"] = 2.0 ** round(math.log2(16.0 / math.sqrt(d)))
    else:
        d = c["d"]
        s["hidden"] = normal(n, d).to(dt)
        s["weight"] = (2.0 / math.sqrt(d) * normal(v, d)).to(dt)
    if c["op"] in ("score_grad", "head_grad"):
        # what the forward pass kept, and the gradient of a mean loss with a small entropy bonus
        x = s["logits"] if c["op"] == "score_grad" else s["hidden"].float() @ s["weight"].float().t()
        x = x.float() * s["scale"]
        s["norm"] = _norm(x)
        lp = (x - s["norm"][:, :1].clamp(min=torch.finfo(torch.float32).min)) - s["norm"][:, 1:]
        s["entropy"] = -(torch.exp(lp) * lp.clamp(min=-1e4)).sum(1)
        s["g_logprob"] = -(0.5 + uniform(n)) / n
        s["g_entropy"] = 0.02 * (uniform(n) - 0.5) / n
    return s


def _plain_score(x, s):
    """Scores from 32-bit logits."""
    m, t = s["case"]["m"], s["targets"].long()
    l = x * s["scale"]
    norm = _norm(l)
    top = norm[:, :1]
    below = l - top.masked_fill(top == -math.inf, 0.0)
    weight = torch.exp(below)
    spread = (weight * below.masked_fill(weight == 0, 0.0)).sum(1) / weight.sum(1)
    entropy = (norm[:, 1] - spread).masked_fill(top[:, 0] == -math.inf, 0.0)
    lp = below - norm[:, 1:]
    logprob = lp.gather(1, t.clamp(min=0)[:, None])[:, 0].masked_fill(t < 0, 0.0)
    if not m:
        return [logprob, entropy, norm]
    # descending by logit, then ascending by index, as one whole number each
    bits = (l + 0.0).view(torch.int32).long()
    key = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF) - 1)
    key = key * 2 ** 31 + (2 ** 31 - 1 - torch.arange(l.shape[1], device=l.device))
    idx = key.topk(m, 1).indices
    top_lp = lp.gather(1, idx)
    idx = idx.to(torch.int32).masked_fill(top_lp == -math.inf, -1)
    return [logprob, entropy, norm, idx, top_lp]


def _plain_dlogits(x, s):
    """Gradient with respect to 32-bit logits."""
    t = s["targets"].long()
    top = s["norm"][:, :1]
    none = top == -math.inf
    lp = (x * s["scale"] - top.masked_fill(none, 0.0)) - s["norm"][:, 1:]
    p = torch.exp(lp)
    g = s["g_logprob"].masked_fill((t < 0) | none[:, 0], 0.0)[:, None]
    dx = -g * p - s["g_entropy"][:, None] * p * (lp.masked_fill(p == 0, 0.0) + s["entropy"][:, None])
    dx.scatter_add_(1, t.clamp(min=0)[:, None], g)
    return dx * s["scale"]


def _plain_moe(s):
    x, m = s["x"].float(), s["case"]["m"]
    f = s["case"]["f"]
    z = x @ s["gate"].float().t()
    bits = (z + 0.0).view(torch.int32).long()
    key = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF) - 1)
    key = key * 2 ** 31 + (2 ** 31 - 1 - torch.arange(z.shape[1], device=z.device))
    idx = key.topk(m, 1).indices
    z = z.gather(1, idx)
    r = torch.exp(z - z[:, :1])
    resp = r / r.sum(1, keepdim=True)
    h = (s["w_in"][idx].float() @ x[:, None, :, None])[..., 0]
    a = h[..., :f] / (1.0 + torch.exp(-h[..., :f])) * h[..., f:]
    y = (s["w_out"][idx].float() @ a[..., None])[..., 0]
    return [(y * resp[..., None]).sum(1).to(s["x"].dtype), idx.to(torch.int32), resp]


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        from gmm_em_amd import ops

        if op == "score":
            return list(ops.logits_score(s["logits"], s["targets"], s["case"]["m"], s["scale"]))
        if op == "score_grad":
            return [ops.logits_score_backward(s["logits"], s["targets"], s["norm"], s["entropy"],
                                              s["g_logprob"], s["g_entropy"], s["scale"])]
        if op == "head":
            return list(ops.head_score(s["hidden"], s["weight"], s["targets"], s["case"]["m"],
                                       s["scale"]))
        if op == "head_grad":
            return list(ops.head_score_backward(s["hidden"], s["weight"], s["targets"], s["norm"],
                                                s["entropy"], s["g_logprob"], s["g_entropy"],
                                                s["scale"]))
        return list(ops.moe_layer(s["x"], s["w_in"], s["w_out"], s["gate"], s["case"]["m"]))
    if op == "score":
        return _plain_score(s["logits"].float(), s)
    if op == "score_grad":
        return [_plain_dlogits(s["logits"].float(), s).to(s["logits"].dtype)]
    if op == "head":
        return _plain_score(s["hidden"].float() @ s["weight"].float().t(), s)
    if op == "head_grad":
        h, w = s["hidden"].float(), s["weight"].float()
        dx = _plain_dlogits(h @ w.t(), s)
        return [(dx @ w).to(s["hidden"].dtype), (dx.t() @ h).to(s["weight"].dtype)]
    return _plain_moe(s)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "moe":
        x, f = s["x"].double(), case["f"]
        z = x @ s["gate"].double().t()
        z, idx = (t[:, :case["m"]] for t in z.sort(dim=1, descending=True, stable=True))
        resp = torch.softmax(z, 1)
        y = torch.zeros_like(x)
        for e in idx.unique().tolist():
            tok, j = (idx == e).nonzero(as_tuple=True)
            h = x[tok] @ s["w_in"][e].double().t()
            a = torch.nn.functional.silu(h[:, :f]) * h[:, f:]
            y.index_add_(0, tok, (a @ s["w_out"][e].double().t()) * resp[tok, j][:, None])
        return [y, None, resp]
    t = s["targets"].long()
    rows = torch.arange(case["n"], device=DEV)
    if "logits" in s:
        l = s["logits"].double() * s["scale"]
    else:
        l = s["hidden"].double() @ s["weight"].double().t() * s["scale"]
    if op in ("score", "head"):
        # rows with nothing left are set apart: their sums say nothing
        empty = (l == -math.inf).all(1)
        lp = torch.log_softmax(l, 1)
        p = lp.exp()
        entropy = -(p * torch.where(p > 0, lp, 0.0)).sum(1)
        entropy[empty] = 0.0
        top = l.amax(1)
        rest = torch.logsumexp(l, 1) - top
        rest[empty] = 0.0
        lp[empty] = -math.inf
        logprob = torch.where(t < 0, 0.0, lp[rows, t.clamp(min=0)])
        out = [logprob, entropy, torch.stack([top, rest], 1)]
        if case["m"]:
            val, at = lp.sort(dim=1, descending=True, stable=True)
            out += [None, val[:, :case["m"]]]
        return out
    top, rest = s["norm"].double().unbind(1)
    empty = top == -math.inf
    lp = l - top[:, None] - rest[:, None]
    lp[empty] = -math.inf
    p = lp.exp()
    hot = torch.zeros_like(p)
    hot[rows, t.clamp(min=0)] = 1.0
    g = torch.where((t < 0) | empty, 0.0, s["g_logprob"].double())
    dl = g[:, None] * (hot - p)
    dl -= s["g_entropy"].double()[:, None] * p * (torch.where(p > 0, lp, 0.0) + s["entropy"].double()[:, None])
    dl *= s["scale"]
    if op == "score_grad":
        return [dl]
    return [dl @ s["weight"].double(), dl.t() @ s["hidden"].double()]
