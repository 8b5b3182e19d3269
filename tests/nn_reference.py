"""Plain float64 forms of the softmax-over-codes operators, from their definitions.

Everything runs in torch float64 on the device of its inputs; nothing of the
library is used.
"""
import torch

INF = float("inf")


def scores(l, targets, m):
    """(logprob, entropy, norm, idx, top) from scaled float64 logits l (N, V)."""
    n, v = l.shape
    empty = (l == -INF).all(1)
    bad = torch.isnan(l).any(1) | (l == INF).any(1)
    top = torch.where(torch.isnan(l), -INF, l).amax(1)
    d = l - torch.where(empty, 0.0, top)[:, None]
    e = torch.where(l == -INF, 0.0, torch.exp(d))
    logs = torch.log(e.sum(1))
    logs[empty] = 0.0
    lp = d - logs[:, None]
    ent = -(torch.exp(lp) * torch.where(l == -INF, 0.0, lp)).sum(1)
    ent[empty] = 0.0
    logs[bad], ent[bad] = float("nan"), float("nan")
    norm = torch.stack([top.masked_fill(bad, float("nan")), logs], 1)
    t = targets.long().clamp(0, v - 1)
    logprob = lp.gather(1, t[:, None])[:, 0]
    logprob[empty] = -INF
    logprob[bad] = float("nan")
    logprob[targets >= v] = float("nan")
    logprob[targets < 0] = 0.0
    key = torch.where(torch.isnan(l), -INF, l)
    val, idx = key.sort(dim=1, descending=True, stable=True)
    val, idx = val[:, :m], idx[:, :m].to(torch.int32)
    lpt = val - top[:, None] - logs[:, None]
    gone = val == -INF
    return logprob, ent, norm, idx.masked_fill(gone, -1), lpt.masked_fill(gone, -INF)


def dlogits(l, targets, g_logprob, g_entropy, scale):
    """Gradient with respect to the unscaled logits, for finite or masked rows."""
    n, v = l.shape
    empty = (l == -INF).all(1)
    _, ent, norm, _, _ = scores(l, targets, 0)
    lp = l - torch.where(empty, 0.0, norm[:, 0])[:, None] - norm[:, 1:]
    p = torch.exp(lp)
    hot = torch.zeros_like(p)
    hot.scatter_(1, targets.long().clamp(min=0)[:, None], 1.0)
    g = torch.where((targets < 0) | empty, 0.0, g_logprob.double())
    d = g[:, None] * (hot - p)
    d -= g_entropy.double()[:, None] * p * (torch.where(p > 0, lp, 0.0) + ent[:, None])
    return scale * d
