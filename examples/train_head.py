"""Trains a small head over R virtual ranks with the operators and the shard
engine together: features -> hidden matrix -> layer norm -> linear head ->
cross entropy.

Two units: the hidden matrix (ZeRO-3: whole at its owner, updated by Muon) and
the norm's scale and offset with the head (FSDP2 shards, updated by AdamW).
Every step gathers both; each rank runs its own batch, its gradients written
straight into its gradient buffers; then the two units are reduced and updated.

    python examples/train_head.py [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fully_sharded_state_gb300 as fsdp  # noqa: E402

IGNORE = -100


def train(steps: int = 60, ranks: int = 4, rows: int = 512, features: int = 256, width: int = 512, vocab: int = 2003,
          masked: float = 0.2, seed: int = 0):
    """The mean loss over the ranks, step by step."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731

    body = fsdp.ShardedUnit([(width, features)], ranks, "zero3", names=["hidden"])
    head = fsdp.ShardedUnit([(width,), (width,), (vocab, width)], ranks, "per_param", names=["gamma", "beta", "head"])
    body.shard_from_full(randn(body.P) / features ** 0.5)
    first = torch.cat([torch.ones(width, device="cuda"), torch.zeros(width, device="cuda"),
                       randn(vocab * width) * 0.02])
    head.shard_from_full(first)
    units = (body, head)
    full = [u.alloc_full() for u in units]
    grads = [u.alloc_grads() for u in units]

    # a fixed teacher gives every rank's batch its targets; some are ignored
    teacher = randn(vocab, features)
    batches = []
    for _ in range(ranks):
        x = randn(rows, features)
        target = (x @ teacher.t()).argmax(1)
        target[torch.rand(rows, device="cuda", generator=gen) < masked] = IGNORE
        batches.append((x.bfloat16(), target))

    muon = fsdp.MuonHP(lr=0.02, momentum=0.9)
    adamw = fsdp.AdamWHP(3e-3, 0.9, 0.99, 1e-8, 0.01)
    losses = []
    for _ in range(steps):
        for u, f in zip(units, full):
            u.all_gather(f)
        total = torch.zeros((), device="cuda")
        for q, (x, target) in enumerate(batches):
            p = body.unflatten(full[0][q]) | head.unflatten(full[1][q])
            g = body.unflatten(grads[0][q]) | head.unflatten(grads[1][q])
            z = x @ p["hidden"].t()
            y, mean, rstd = fsdp.layer_norm(z, p["gamma"], p["beta"])
            loss, _, dy, _ = fsdp.linear_cross_entropy_grad(y, p["head"], target, ignore_index=IGNORE,
                                                            dweight=g["head"])
            dz, _, _ = fsdp.layer_norm_backward(dy, z, p["gamma"], mean, rstd, dgamma=g["gamma"], dbeta=g["beta"])
            torch.matmul(dz.t(), x, out=g["hidden"])
            total += loss
        body.reduce_scatter_muon(grads[0], muon)
        head.reduce_scatter_adamw(grads[1], adamw)
        losses.append(total / ranks)
    return [float(v) for v in torch.stack(losses)]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    for i, v in enumerate(train(a.steps)):
        if i % 10 == 0 or i + 1 == a.steps:
            print(f"step {i:4d}  loss {v:.4f}")
