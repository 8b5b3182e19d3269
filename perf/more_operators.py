"""The library's operators for sequences of codes as cases to be measured.

Four groups: the embedding of codes and its gradient, the product with 8-bit weights (rows are
quantised in the call), a step of beam search with the states that follow it, and the balance loss of a
router with its gradient. ``run`` makes the calls of ``gmm_em_amd.ops`` where ``own`` is true and computes
the same in plain torch operations where it is not; ``exact`` computes it in 64 bits from the definitions.

Logits whose order decides an output lie on a grid, as those of 8-bit heads nearly do, and the beams'
scores are drawn again where the continuations of two beams are nearer than rounding can tell apart.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
END = 1  # the code that ends a sequence


def listed():
    return [
        # a decoding step: the codes that 32 beams chose last, of the wide workload's 768 dims and 16384 codes
        {"name": "embed_decode", "op": "embed", "n": 32, "d": 768, "v": 16384, "dtype": "bf16"},
        # a training batch's codes, odd in every direction
        {"name": "embed_batch_odd", "op": "embed", "n": 20011, "d": 1001, "v": 40009, "dtype": "f32"},
        # gradient of a small ragged batch
        {"name": "embed_grad_odd", "op": "embed_grad", "n": 257, "d": 100, "v": 1001, "dtype": "f32"},
        # gradient of a training batch whose codes are met with uneven frequency
        {"name": "embed_grad_batch", "op": "embed_grad", "n": 65536, "d": 768, "v": 16384, "dtype": "bf16"},
        # one row through an 8-bit head: latency
        {"name": "int8_one_row", "op": "int8", "n": 1, "d": 768, "v": 16384, "dtype": "bf16"},
        # a prompt's rows, odd in every direction, fp32 in and out
        {"name": "int8_prompt_odd", "op": "int8", "n": 777, "d": 1003, "v": 5001, "dtype": "f32"},
        # a batch of a wide layer
        {"name": "int8_batch", "op": "int8", "n": 8192, "d": 4096, "v": 16384, "dtype": "bf16"},
        # the first step of four searches: one beam becomes eight
        {"name": "beam_first", "op": "beam", "b": 4, "w": 1, "m": 8, "v": 16384, "dtype": "f32", "masked": False,
         "layers": 2, "t": 1, "d": 96},
        # a later step with a grammar mask, some beams ended, some dead; odd sizes
        {"name": "beam_masked_odd", "op": "beam", "b": 7, "w": 5, "m": 5, "v": 40009, "dtype": "f32",
         "masked": True, "layers": 3, "t": 37, "d": 100},
        # a batch of searches with wide beams
        {"name": "beam_batch", "op": "beam", "b": 64, "w": 16, "m": 16, "v": 32768, "dtype": "bf16",
         "masked": False, "layers": 4, "t": 64, "d": 128},
        # the router of a small padded batch
        {"name": "balance_odd", "op": "balance", "n": 333, "e": 60, "m": 2, "dtype": "f32"},
        # the router of a training batch
        {"name": "balance_batch", "op": "balance", "n": 65536, "e": 128, "m": 8, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "int8", "beam", "balance"])
    c = {"op": op, "dtype": rng.choice(["f32", "bf16"])}
    es = SIZE[c["dtype"]]
    if op in ("embed", "embed_grad"):
        c["n"], c["d"], c["v"] = _log(rng, 1, 65536), _log(rng, 32, 2048), _log(rng, 100, 65536)
        # what is read and written is at most the listed batch's
        most = (65536 + 16384) * 768 * 2
        c["d"] = max(8, min(c["d"], most // (es * (c["n"] + c["v"]))))
    elif op == "int8":
        c["n"], c["d"], c["v"] = _log(rng, 1, 8192), _log(rng, 32, 8192), _log(rng, 100, 32768)
        c["n"] = max(1, min(c["n"], 8192 * 4096 * 16384 // (c["d"] * c["v"]), 8192 * 4096 * 10 // (es * (c["d"] + c["v"]))))
    elif op == "beam":
        c["w"], c["v"] = rng.choice([1, rng.randint(2, 8), rng.randint(2, 16)]), _log(rng, 100, 65536)
        c["m"] = rng.randint(1, 16) if c["w"] == 1 else c["w"]
        c["b"] = max(1, min(_log(rng, 1, 64), 64 * 16 * 32768 * 2 // (es * c["w"] * c["v"])))
        c["masked"] = rng.random() < 0.5
        c["layers"], c["t"], c["d"] = rng.randint(1, 4), _log(rng, 1, 64), _log(rng, 16, 128)
    else:
        c["n"], c["e"] = _log(rng, 1, 65536), _log(rng, 4, 512)
        c["n"] = max(1, min(c["n"], 65536 * 128 * 2 // (es * c["e"])))
        c["m"] = rng.randint(1, min(8, c["e"]))
    return c


def work(case):
    c, es = case, SIZE[case["dtype"]]
    if c["op"] == "embed":
        distinct = c["v"] * (1.0 - (1.0 - 1.0 / c["v"]) ** c["n"])
        return {"bytes": int((c["n"] + distinct) * c["d"] * es) + 4 * c["n"], "flops": 1.0 * c["n"] * c["d"]}
    if c["op"] == "embed_grad":
        return {"bytes": (c["n"] + c["v"]) * c["d"] * es + 4 * c["n"], "flops": 1.0 * c["n"] * c["d"]}
    if c["op"] == "int8":
        n, d, v = c["n"], c["d"], c["v"]
        return {"bytes": n * d * es + v * d + 4 * (n + v) + n * v * es, "flops": 2.0 * n * d * v}
    if c["op"] == "beam":
        rows, out = c["b"] * c["w"], c["b"] * c["m"]
        state = c["layers"] * c["t"] * c["d"] * 2 + 4 * c["t"]
        return {"bytes": rows * c["v"] * es + 8 * rows + 12 * out + out * 2 * state,
                "flops": 4.0 * rows * c["v"]}
    return {"bytes": 2 * c["n"] * c["e"] * es + 4 * c["n"] * c["m"], "flops": 10.0 * c["n"] * c["e"]}


def _spread(s, l, uniform):
    """Scores of the beams (B, W), drawn so that no two beams' continuations are too near to be ranked."""
    c = s["case"]
    b, w, m = c["b"], c["w"], c["m"]
    top = l.amax(1, keepdim=True)
    none = top == -math.inf
    norm = top.masked_fill(none, 0.0) + torch.exp(l - top.masked_fill(none, 0.0)).sum(1, keepdim=True).log()
    best = (l.topk(min(m + 1, c["v"]), 1).values - norm).masked_fill(none, -math.inf)
    ended = s["last"].view(-1, 1) == END
    best = best.masked_fill(ended, -math.inf)
    best[:, 0] = best[:, 0].masked_fill(ended[:, 0], 0.0)  # an ended beam goes on as itself
    best = best.view(b, w, -1)
    beam = torch.arange(w, device=DEV)[:, None].expand(w, best.shape[2]).reshape(-1)
    scores = torch.zeros(b, w, device=DEV)
    redo = torch.ones(b, dtype=torch.bool, device=DEV)
    dead = uniform(b, w) < (0.1 if c["masked"] and w > 1 else 0.0)  # beams that never were
    for _ in range(20):
        drawn = -2.0 - 6.0 * uniform(b, w)
        scores = torch.where(redo[:, None], drawn, scores).masked_fill(dead, -math.inf)
        cand, at = (best + scores.double()[:, :, None]).view(b, -1).sort(dim=1, descending=True, stable=True)
        gap = cand[:, :-1] - cand[:, 1:]
        redo = ((gap < 2e-4) & (beam[at[:, :-1]] != beam[at[:, 1:]]))[:, :m + 1].any(1)
    return scores


def prepare(case, seed):
    c, dt = case, TYPES[case["dtype"]]
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    s = {"case": dict(c)}
    if c["op"] in ("embed", "embed_grad"):
        n, d, v = c["n"], c["d"], c["v"]
        # codes are met with uneven frequency; some places are padding
        s["codes"] = (v * uniform(n) ** 3).to(torch.int32).clamp_(max=v - 1)
        s["codes"][uniform(n) < 0.05] = -1
        s["scale"] = math.sqrt(d)
        s["x"] = (normal(v, d) / math.sqrt(d) if c["op"] == "embed" else normal(n, d) / n).to(dt)
        return s
    if c["op"] == "int8":
        n, d, v = c["n"], c["d"], c["v"]
        # activations have a few wide dims; weights come quantised from the program that loaded them
        s["x"] = (normal(n, d) * torch.exp(0.5 * normal(d))).to(dt)
        w = normal(v, d) * (0.5 + uniform(v, 1)) / math.sqrt(d)
        s["w_scale"] = w.abs().amax(1) / 127.0
        s["w"] = torch.round(w / s["w_scale"][:, None]).clamp_(-127, 127).to(torch.int8)
        return s
    if c["op"] == "balance":
        n, e, m = c["n"], c["e"], c["m"]
        z = 1.5 * normal(n, e) + normal(e)  # some experts are favoured
        s["idx"] = z.topk(m, 1).indices.to(torch.int32)
        s["idx"][uniform(n) < 0.1] = -1     # padding is not routed
        s["z"] = z.to(dt)
        s["g"] = torch.full((), 0.01, device=DEV)
        return s
    rows, v, t = c["b"] * c["w"], c["v"], c["t"]
    x = (2.5 * normal(rows, v) * 16.0).round_().clamp_(-255, 255) / 16.0
    if c["masked"]:
        x[uniform(rows, v) < 0.3] = -math.inf
        x[uniform(rows) < 0.1] = -math.inf  # beams with no code left
    s["logits"] = x.to(dt)
    s["scale"] = 1.25  # a temperature of 0.8
    s["last"] = (v * uniform(c["b"], c["w"])).to(torch.int32).clamp_(min=2, max=v - 1)
    if c["w"] > 1:
        s["last"][uniform(c["b"], c["w"]) < 0.1] = END
    s["scores"] = _spread(s, s["logits"].double() * s["scale"], uniform)
    s["history"] = (v * uniform(rows, t)).to(torch.int32)
    s["cache"] = normal(c["layers"], rows, t, c["d"]).to(torch.bfloat16)
    return s


def _plain_beam(s):
    c = s["case"]
    b, w, m, v = c["b"], c["w"], c["m"], c["v"]
    l = s["logits"].float() * s["scale"]
    top = l.amax(1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    lp = (l - top) - torch.exp(l - top).sum(1, keepdim=True).log()
    ended = (s["last"] == END).view(-1, 1)
    code = torch.arange(v, device=DEV)
    lp = torch.where(ended, torch.where(code == END, 0.0, -math.inf), lp).masked_fill(
        (l == -math.inf) & ~ended, -math.inf)
    score = (s["scores"].view(-1, 1) + lp).view(b, w * v)
    # descending by score, then ascending by beam and code, as one whole number each
    bits = (score + 0.0).view(torch.int32).long()
    key = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF) - 1)
    key = key * 2 ** 31 + (2 ** 31 - 1 - torch.arange(w * v, device=DEV))
    at = key.topk(m, 1).indices
    score = score.gather(1, at)
    none = score == -math.inf
    parent = (at // v).masked_fill(none, -1)
    row = parent.clamp(min=0) + w * torch.arange(b, device=DEV)[:, None]
    gone = none.view(-1)
    history = s["history"][row.view(-1)].masked_fill(gone[:, None], 0)
    cache = s["cache"][:, row.view(-1)].masked_fill(gone[:, None, None], 0.0)
    return [parent.to(torch.int32), (at % v).masked_fill(none, -1).to(torch.int32), score, history, cache]


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        from gmm_em_amd import ops

        if op == "embed":
            return [ops.embed(s["x"], s["codes"], s["scale"])]
        if op == "embed_grad":
            return [ops.embed_backward(s["x"], s["codes"], s["case"]["v"], s["scale"])]
        if op == "int8":
            q, scale = ops.quantize_rows(s["x"])
            return [ops.quantized_product(q, scale, s["w"], s["w_scale"], s["x"].dtype), scale]
        if op == "balance":
            r = ops.balance_loss(s["z"], s["idx"])
            dz = ops.balance_loss_backward(s["z"], r.counts, r.totals, r.norm, s["g"])
            return [r.loss, r.counts, r.prob, dz]
        r = ops.beam_step(s["logits"], s["scores"], s["last"], END, s["case"]["m"], s["scale"])
        return [r.parent, r.code, r.score, ops.beam_reorder(s["history"], r.parent, s["case"]["w"]),
                ops.beam_reorder(s["cache"], r.parent, s["case"]["w"], dim=1)]
    if op == "embed":
        t = s["codes"].long()
        out = s["x"][t.clamp(min=0)].float() * s["scale"]
        return [out.masked_fill((t < 0)[:, None], 0.0).to(s["x"].dtype)]
    if op == "embed_grad":
        t = s["codes"].long()
        g = s["x"].float().masked_fill((t < 0)[:, None], 0.0)
        out = torch.zeros(s["case"]["v"], g.shape[1], device=DEV).index_add_(0, t.clamp(min=0), g)
        return [(out * s["scale"]).to(s["x"].dtype)]
    if op == "int8":
        x = s["x"].float()
        scale = (x.abs().amax(1).double() / 127.0).float()
        # next to a border 64 bits tell the nearest integer
        q = torch.round(x.double() / scale.double()[:, None]).float()
        y = (q @ s["w"].float().t()) * (scale[:, None] * s["w_scale"])
        return [y.to(s["x"].dtype), scale]
    if op == "balance":
        n, e = s["case"]["n"], s["case"]["e"]
        live = s["idx"][:, 0] >= 0
        counts = torch.zeros(e + 1, dtype=torch.int64, device=DEV)
        counts.scatter_add_(0, s["idx"].view(-1).long() % (e + 1), torch.ones_like(s["idx"].view(-1).long()))
        counts = counts[:e]
        z = s["z"].float()
        p = torch.exp(z - z.amax(1, keepdim=True))
        p = (p / p.sum(1, keepdim=True)).masked_fill(~live[:, None], 0.0)
        rows = live.sum().clamp(min=1)
        f = counts.float() / counts.sum().clamp(min=1)
        prob = p.sum(0) / rows
        dz = s["g"] * e / rows * p * (f - (p @ f)[:, None])
        return [e * (f * prob).sum(), counts.to(torch.int32), prob, dz.to(s["z"].dtype)]
    return _plain_beam(s)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        keep = (s["codes"] >= 0).double()[:, None]
        return [torch.nn.functional.embedding(s["codes"].long().clamp(min=0), s["x"].double()) * keep * s["scale"]]
    if op == "embed_grad":
        order = s["codes"].long().argsort(stable=True)
        order = order[s["codes"][order] >= 0]
        out = torch.zeros(case["v"], case["d"], dtype=torch.float64, device=DEV)
        # running sums of the sorted rows, a stretch of dims at a time
        ends = torch.searchsorted(s["codes"][order].long(), torch.arange(case["v"] + 1, device=DEV))
        for k in range(0, case["d"], 64):
            run_ = torch.cumsum(s["x"][order, k:k + 64].double(), 0)
            run_ = torch.cat([torch.zeros_like(out[:1, k:k + 64]), run_])
            out[:, k:k + 64] = run_[ends[1:]] - run_[ends[:-1]]
        out[ends[1:] == ends[:-1]] = 0.0
        return [out * s["scale"]]
    if op == "int8":
        x = s["x"].double()
        scale = x.abs().amax(1) / 127.0
        q = torch.round(x / scale.float().double()[:, None])
        y = q @ s["w"].double().t()
        y *= scale.float().double()[:, None]
        y *= s["w_scale"].double()
        return [y, scale]
    if op == "balance":
        live = s["idx"][:, 0] >= 0
        p = torch.softmax(s["z"].double(), 1)[live]
        f = torch.bincount(s["idx"][live].view(-1), minlength=case["e"]).double()
        f /= max(1.0, float(f.sum()))
        rows = max(1, p.shape[0])
        prob = p.sum(0) / rows
        dz = torch.zeros(case["n"], case["e"], dtype=torch.float64, device=DEV)
        dz[live] = p * (f - p @ f[:, None]) * (case["e"] / rows) * s["g"].double()
        return [case["e"] * torch.dot(f, prob), None, prob, dz]
    b, w, m, v = case["b"], case["w"], case["m"], case["v"]
    lp = s["logits"].double() * s["scale"]
    empty = (lp == -math.inf).all(1)
    lp = torch.log_softmax(lp, 1)
    lp[empty] = -math.inf
    ended = (s["last"] == END).view(-1)
    lp[ended] = -math.inf
    lp[ended, END] = 0.0
    lp += s["scores"].double().view(-1, 1)
    score, at = lp.view(b, w * v).sort(dim=1, descending=True, stable=True)
    score, at = score[:, :m], at[:, :m]
    row = (at // v + w * torch.arange(b, device=DEV)[:, None]).view(-1)
    cache = s["cache"].double()[:, row]
    cache[:, (score == -math.inf).view(-1)] = 0.0
    return [None, None, score, None, cache]
