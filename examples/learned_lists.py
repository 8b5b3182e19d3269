"""Inverted lists from a learned softmax over codes, instead of from the mixture itself.

Rows are quantised to codes by k-means. A head (one weight row per code) learns
to predict a row's code; its two most probable codes and their probabilities then fill
the inverted lists, in place of the mixture's soft assignments. At query time a few
rows pass through a mixture-of-experts layer, routed by a Gaussian mixture, and
their logits are scored for the lists to visit.

Run on an MI355X: python examples/learned_lists.py
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gmm_em_amd import datagen as dg  # noqa: E402
from gmm_em_amd import ops  # noqa: E402


def train_head(h, codes, k, steps, lr):
    """Gradient descent on the mean of -log p(code); returns (weight, losses)."""
    n, d = h.shape
    weight = torch.zeros(k, d, dtype=h.dtype, device=h.device)
    master = weight.float()
    g = torch.full((n,), -1.0 / n, device=h.device)
    losses = []
    for _ in range(steps):
        s = ops.head_score(h, weight, codes)
        losses.append(-s.logprob.mean())
        _, dw = ops.head_score_backward(h, weight, codes, s.norm, s.entropy, g)
        master -= lr * dw.float()
        weight = master.to(h.dtype)
    return weight, torch.stack(losses).tolist()


def main(n: int = 20_000, k: int = 256, steps: int = 40, experts: int = 8, seed: int = 0):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    work = dg.WORKLOADS["descriptor"]
    x = torch.from_numpy(dg.rows(work, n)).to(dev)
    d = x.shape[1]

    # codes of the rows
    pick = torch.randperm(n, generator=gen, device=dev)
    centroids = x[pick[:k]].clone()
    ops.kmeans_fit(x, centroids, max_iter=5)
    _, codes = ops.kmeans_step(x, centroids.clone())

    # a head that predicts them, in bf16
    h = ((x - x.mean(0)) / x.std(0).clamp(min=1.0)).to(torch.bfloat16)
    weight, losses = train_head(h, codes, k, steps, lr=0.3)

    # each row into its most probable code's list, border rows into the second's too
    s = ops.head_score(h, weight, codes, m=2)
    offsets, rows, values = ops.ivf_build(s.top_idx, s.top_logprob.exp(), k, 0.1)
    agree = (s.top_idx[:, 0] == codes).float().mean().item()

    # a few query rows: experts picked by a mixture's responsibilities, then the lists to visit
    q = h[:4].contiguous()
    w = torch.full((experts,), 1.0 / experts, device=dev)
    mu = h[pick[k:k + experts]].float()
    var = torch.ones(experts, d, device=dev)
    idx, resp = ops.assign_topm(q.float(), w, mu, var, m=2)
    f = 2 * d
    w_in = (torch.randn(experts, 2 * f, d, generator=gen, device=dev) / d ** 0.5).to(torch.bfloat16)
    w_out = (0.1 * torch.randn(experts, d, f, generator=gen, device=dev) / f ** 0.5).to(torch.bfloat16)
    y, _, _ = ops.moe_layer(q, w_in, w_out, idx=idx, resp=resp)
    refined = q + y
    logits = refined.float() @ weight.float().t()
    visit = ops.logits_score(logits, codes[:4].contiguous(), m=4)
    # the gradient that would reach the experts through the logits, in place of them
    ops.logits_score_backward(logits, codes[:4].contiguous(), visit.norm, visit.entropy,
                              torch.full((4,), -0.25, device=dev), out=logits)
    d_refined = logits @ weight.float()

    out = {"losses": losses, "agree": agree, "entries": int(rows.numel()),
           "entropy": s.entropy.mean().item(), "visit": visit.top_idx.cpu(),
           "offsets": offsets.cpu(), "rows": rows.cpu(), "d_refined": d_refined.cpu()}
    print(f"rows {n}, codes {k}: loss {losses[0]:.3f} -> {losses[-1]:.3f}, "
          f"most probable code is the row's own for {100 * agree:.1f} %, "
          f"{out['entries'] / n:.2f} lists a row, mean entropy {out['entropy']:.3f}")
    return out


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rows", type=int, default=20_000)
    ap.add_argument("--codes", type=int, default=256)
    ap.add_argument("--steps", type=int, default=40)
    a = ap.parse_args()
    main(a.rows, a.codes, a.steps)
