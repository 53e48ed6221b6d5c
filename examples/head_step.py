"""Trains a language model's head for a few steps: the last norm, the
classifier with its cross entropy, the backward pass, clipping and an update.

    python examples/head_step.py [--norm layer|rms] [--steps 20] [--tokens 1024]

The hidden states are fixed synthetic ones in a 32-bit residual stream, whose
norm is the 16-bit input of the classifier.  Needs a GB300 and the built
library.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import linear_cross_entropy_gb300 as cce  # noqa: E402


class Head(torch.nn.Module):
    """norm -> linear -> cross entropy, with fp32 norm parameters and a bf16 classifier."""

    def __init__(self, dim, vocab, norm="layer", device="cuda"):
        super().__init__()
        self.norm = norm
        self.weight = torch.nn.Parameter(torch.ones(dim, device=device))
        self.bias = torch.nn.Parameter(torch.zeros(dim, device=device)) if norm == "layer" else None
        self.classifier = torch.nn.Parameter((torch.randn(vocab, dim, device=device) / dim ** 0.5).bfloat16())

    def forward(self, hidden, targets):
        """hidden [..., dim] fp32 or bf16, targets [...] int64; rows with target -100 take no part."""
        if self.norm == "layer":
            e = cce.layer_norm(hidden, self.weight, self.bias, out_dtype=torch.bfloat16)
        else:
            e = cce.rms_norm(hidden, self.weight, out_dtype=torch.bfloat16)
        return cce.linear_cross_entropy(e.view(-1, e.shape[-1]), self.classifier, targets.reshape(-1))


def train(norm="layer", steps=20, tokens=1024, dim=128, vocab=4096, lr=0.5, max_norm=1.0, seed=0):
    """The losses and the gradient norms of the steps."""
    torch.manual_seed(seed)
    head = Head(dim, vocab, norm)
    hidden = torch.randn(4, tokens // 4, dim, device="cuda") * 3 + 0.5
    targets = torch.randint(0, vocab, (4, tokens // 4), device="cuda")
    # every position predicts the next one: the last of each sequence has no target
    hidden, targets = hidden[:, :-1], targets[:, 1:]
    losses, norms = [], []
    for _ in range(steps):
        loss = head(hidden, targets)
        head.zero_grad(set_to_none=True)
        loss.backward()
        norms.append(cce.clip_grad_norm_(head.parameters(), max_norm))
        with torch.no_grad():
            for p in head.parameters():
                p.sub_(p.grad, alpha=lr)
        losses.append(loss.detach())
    cce.raise_pending_errors()
    return [float(v) for v in losses], [float(v) for v in norms]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--norm", choices=("layer", "rms"), default="layer")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=1024)
    a = ap.parse_args()
    for i, (loss, norm) in enumerate(zip(*train(a.norm, a.steps, a.tokens))):
        print(f"step {i:3d}  loss {loss:.4f}  gradient norm {norm:.4f}")


if __name__ == "__main__":
    main()
