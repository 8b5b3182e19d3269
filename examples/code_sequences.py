"""Sequences of codes from a learned model, by beam search on an 8-bit head.

Rows are quantised twice by k-means, the second time what the first code leaves of them, so that a
row's name is a sequence of two codes and an end. A model reads a row and the codes so far (their
embeddings are added) and predicts the next code; its embedding and head are trained on the log-probabilities,
and a gate over experts on its balance loss. Then query rows pass through the experts that the gate picks,
and beam search over the head in 8 bits gives the most probable sequences: the lists to visit.

Run on an MI355X: python examples/code_sequences.py
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gmm_em_amd import datagen as dg  # noqa: E402
from gmm_em_amd import ops  # noqa: E402

START, END = 0, 1  # codes 2 .. k + 1 name the first level, k + 2 .. 2 k + 1 the second


def sequences(x, k, gen):
    """(N, 4) int32: the start, a code of each level and the end."""
    n = x.shape[0]
    seq = torch.full((n, 4), END, dtype=torch.int32, device=x.device)
    seq[:, 0] = START
    left = x.clone()
    for level in range(2):
        pick = torch.randperm(n, generator=gen, device=x.device)[:k]
        centroids = left[pick].clone()
        ops.kmeans_fit(left, centroids, max_iter=5)
        _, z = ops.kmeans_step(left, centroids.clone())
        left -= centroids[z.long()]
        seq[:, 1 + level] = z + (2 + level * k)
    return seq


def train(h, seq, v, steps, lr):
    """Gradient descent on the mean of -log p(next code): (table, head, losses), in h's type."""
    n, d = h.shape
    dev = h.device
    table, head = (torch.zeros(v, d, device=dev) for _ in range(2))
    g = torch.full((n,), -1.0 / n, device=dev)
    losses = []
    for _ in range(steps):
        low_table, low_head = table.to(h.dtype), head.to(h.dtype)
        hidden, loss = h, torch.zeros((), device=dev)
        d_state = torch.zeros(n, d, device=dev)
        grads = []
        for t in range(3):
            hidden = hidden + ops.embed(low_table, seq[:, t].contiguous())
            target = seq[:, t + 1].contiguous()
            s = ops.head_score(hidden, low_head, target)
            dh, dw = ops.head_score_backward(hidden, low_head, target, s.norm, s.entropy, g)
            loss -= s.logprob.mean()
            head -= lr * dw.float()
            grads.append(dh)
        # a code's embedding is part of every state after it
        for t in reversed(range(3)):
            d_state += grads[t].float()
            table -= lr * ops.embed_backward(d_state, seq[:, t].contiguous(), v)
        losses.append(loss / 3)
    return table.to(h.dtype), head.to(h.dtype), torch.stack(losses).tolist()


def train_gate(h, gate, m, steps, lr):
    """The gate moved along its balance loss: (gate, losses)."""
    losses = []
    for _ in range(steps):
        z = h.float() @ gate.t()
        r = ops.balance_loss(z, z.topk(m, 1).indices.to(torch.int32))
        dz = ops.balance_loss_backward(z, r.counts, r.totals, r.norm)
        gate = gate - lr * dz.t() @ h.float()
        losses.append(r.loss)
    return gate, torch.stack(losses).tolist()


def step_mask(k, v, t, dev):
    """Codes that step t may not choose."""
    off = torch.ones(v, dtype=torch.bool, device=dev)
    if t < 2:
        off[2 + t * k:2 + (t + 1) * k] = False
    else:
        off[END] = False
    return off


def decode_step(hidden, head, head_scale, off, scores, last, w):
    """One step: the 8-bit head's logits, the grammar's mask, the best continuations."""
    logits = ops.quantized_product(*ops.quantize_rows(hidden), head, head_scale, torch.float32)
    logits.masked_fill_(off, float("-inf"))
    return ops.beam_step(logits, scores, last, END, w), logits


def search(hidden, table, head, head_scale, k, w):
    """Beam search for each row of hidden (B, D): codes (B, w, 3) and scores (B, w)."""
    b = hidden.shape[0]
    dev, v = hidden.device, table.shape[0]
    scores = torch.zeros(b, 1, device=dev)
    last = torch.full((b, 1), START, dtype=torch.int32, device=dev)
    history = torch.empty(b, 0, dtype=torch.int32, device=dev)
    hidden = hidden + ops.embed(table, last.view(-1))
    for t in range(3):
        beams, _ = decode_step(hidden, head, head_scale, step_mask(k, v, t, dev), scores, last, w)
        wide = scores.shape[1]
        hidden = ops.beam_reorder(hidden, beams.parent, wide)
        history = torch.cat([ops.beam_reorder(history, beams.parent, wide), beams.code.view(-1, 1)], 1)
        scores, last = beams.score, beams.code
        hidden = hidden + ops.embed(table, last.view(-1))
    return history.view(b, w, 3), scores


def main(n: int = 20_000, k: int = 64, steps: int = 40, queries: int = 64, w: int = 4, seed: int = 0):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    x = torch.from_numpy(dg.rows(dg.WORKLOADS["descriptor"], n)).to(dev)
    d, v = x.shape[1], 2 + 2 * k
    seq = sequences(x, k, gen)
    h = ((x - x.mean(0)) / x.std(0).clamp(min=1.0)).to(torch.bfloat16)
    table, head, losses = train(h, seq, v, steps, lr=0.3)

    experts, m, f = 8, 2, 2 * d
    gate = torch.randn(experts, d, generator=gen, device=dev) / d ** 0.5
    gate, balance = train_gate(h, gate, m, 20, lr=1.0)

    # serving: experts of the gate's choice, the head in 8 bits
    q = h[:queries].contiguous()
    w_in = (torch.randn(experts, 2 * f, d, generator=gen, device=dev) / d ** 0.5).to(h.dtype)
    w_out = (0.02 * torch.randn(experts, d, f, generator=gen, device=dev) / f ** 0.5).to(h.dtype)
    y, _, _ = ops.moe_layer(q, w_in, w_out, gate.to(h.dtype), m)
    low, low_scale = ops.quantize_rows(head)
    found, scores = search(q + y, table, low, low_scale, k, w)

    own = (found[:, :, :2] == seq[:queries, None, 1:3]).all(2).any(1).float().mean().item()
    print(f"rows {n}, codes {k} x 2: loss {losses[0]:.3f} -> {losses[-1]:.3f}, balance {balance[0]:.3f} -> "
          f"{balance[-1]:.3f}, the row's own sequence is among the {w} best for {100 * own:.1f} %")
    return {"losses": losses, "balance": balance, "found": found, "scores": scores, "own": own, "q": q + y,
            "table": table, "head": low, "head_scale": low_scale, "k": k, "w": w, "seq": seq}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rows", type=int, default=20_000)
    ap.add_argument("--codes", type=int, default=64)
    ap.add_argument("--steps", type=int, default=40)
    a = ap.parse_args()
    main(a.rows, a.codes, a.steps)
