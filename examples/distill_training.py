"""A small model around the MoE layer, trained by distillation.

Token embedding, two MoE blocks between block norms (the residual stream in
float32, each block behind a learned gate for every channel), logits from the
embedding's own table, and the distillation loss against a teacher known by
its top logits; every operator but the logits' matrix product is the
library's.  Runs on a GB300:

    python examples/distill_training.py [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import top_routed_grouped_gb300 as moe  # noqa: E402


class Trunk(torch.nn.Module):
    """ids [T] -> logits [T, V]."""

    def __init__(self, vocabulary: int, hidden: int, blocks: int, experts: int, top_k: int, intermediate: int):
        super().__init__()
        self.embedding = moe.TokenEmbedding(vocabulary, hidden, scale=hidden ** 0.5, out_dtype=torch.float32)
        self.first = moe.BlockNorm(hidden, post=False)
        self.blocks = torch.nn.ModuleList(
            moe.MoELayer(hidden, experts, top_k, intermediate, intermediate) for _ in range(blocks))
        self.joins = torch.nn.ModuleList(moe.BlockNorm(hidden) for _ in range(blocks))
        self.gates = torch.nn.ParameterList(
            torch.nn.Parameter(torch.full((hidden,), 0.5, dtype=torch.bfloat16, device="cuda")) for _ in range(blocks))

    def forward(self, ids: torch.Tensor) -> torch.Tensor:
        r = self.embedding(ids)
        h = self.first(r, dtype=torch.bfloat16)
        for block, join, gate in zip(self.blocks, self.joins, self.gates):
            r, h = join(r, block(h), gate)
        return h @ self.embedding.weight.t()


def train(steps: int = 20, tokens: int = 512, vocabulary: int = 8000, hidden: int = 256, slots: int = 16,
          seed: int = 0) -> list[float]:
    """Losses of ``steps`` steps on one batch with a random teacher."""
    torch.manual_seed(seed)
    model = Trunk(vocabulary, hidden, blocks=2, experts=16, top_k=4, intermediate=256)
    optimizer = torch.optim.AdamW(model.parameters(), lr=2e-3, weight_decay=0.0)
    ids = torch.randint(vocabulary, (tokens,), device="cuda")
    t_ids = torch.rand(tokens, vocabulary, device="cuda").topk(slots, dim=1).indices.int()
    t_logits = 2 * torch.randn(tokens, slots, device="cuda")
    t_ids[: tokens // 8] = -1  # a prompt: no teacher there
    losses = []
    for _ in range(steps):
        loss = moe.distillation_loss(model(ids), t_ids, t_logits, temperature=1.0).mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(float(loss.detach()))
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    for i, v in enumerate(train(ap.parse_args().steps)):
        print(f"step {i}: loss {v:.4f}")
