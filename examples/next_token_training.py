"""A small model around the MoE layer, trained on the next token.

The trunk of ``distill_training.py`` (token embedding, two MoE blocks between
block norms), whose last rows go straight into the cross entropy of the next
token against the embedding's own table: no logits are kept.  The gradients'
global norm is clipped before each update.  Runs on a GB300:

    python examples/next_token_training.py [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import top_routed_grouped_gb300 as moe  # noqa: E402
from distill_training import Trunk  # noqa: E402


class Model(Trunk):
    """ids [T], targets [T] -> loss [T]."""

    def __init__(self, vocabulary: int, hidden: int, **kw):
        super().__init__(vocabulary, hidden, **kw)
        self.head = moe.LMHead(vocabulary, hidden, z_loss=1e-4, weight=self.embedding.weight)

    def forward(self, ids: torch.Tensor, targets: torch.Tensor) -> torch.Tensor:
        r = self.embedding(ids)
        h = self.first(r, dtype=torch.bfloat16)
        for block, join, gate in zip(self.blocks, self.joins, self.gates):
            r, h = join(r, block(h), gate)
        return self.head(h, targets)


def train(steps: int = 20, tokens: int = 512, vocabulary: int = 8000, hidden: int = 256, max_norm: float = 1.0,
          seed: int = 0) -> tuple[list[float], list[float]]:
    """Losses and gradient norms of ``steps`` steps on one random sequence."""
    torch.manual_seed(seed)
    model = Model(vocabulary, hidden, blocks=2, experts=16, top_k=4, intermediate=256)
    optimizer = torch.optim.AdamW(model.parameters(), lr=2e-3, weight_decay=0.0)
    ids = torch.randint(vocabulary, (tokens + 1,), device="cuda")
    targets = ids[1:].clone()
    targets[: tokens // 8] = -100  # a prompt: nothing to learn there
    count = int((targets >= 0).sum())
    losses, norms = [], []
    for _ in range(steps):
        loss = model(ids[:-1], targets).sum() / count
        optimizer.zero_grad()
        loss.backward()
        norms.append(float(moe.clip_grad_norm_(model.parameters(), max_norm)))
        optimizer.step()
        losses.append(float(loss.detach()))
    return losses, norms


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    for i, (loss, norm) in enumerate(zip(*train(ap.parse_args().steps))):
        print(f"step {i}: loss {loss:.4f}, gradient norm {norm:.3f}")
