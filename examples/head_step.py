"""Trains a language model's head for a few steps: the last norm, the
classifier with its cross entropy, the backward pass, clipping and an update.

    python examples/head_step.py [--norm layer|rms] [--steps 20] [--tokens 1024]
                                 [--block none|transform|gated] [--optimizer sgd|adamw|adamw8]

The hidden states are fixed synthetic ones in a 32-bit residual stream, whose
norm is the 16-bit input of the classifier.  With --block a layer comes before
that norm: the dense transform of a masked-language-model head, or a gated
feed-forward block with its residual.  With AdamW the gradients are clipped on the
way of the update (states in 32 or in 8 bits, fp32 master weights).  Needs a GB300
and the built library.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import linear_cross_entropy_gb300 as cce  # noqa: E402


class Transform(torch.nn.Module):
    """gelu(W x + b) on the 16-bit hidden states, as 32-bit ones."""

    def __init__(self, dim, device="cuda"):
        super().__init__()
        self.weight = torch.nn.Parameter((torch.randn(dim, dim, device=device) / dim ** 0.5).bfloat16())
        self.bias = torch.nn.Parameter(torch.zeros(dim, device=device, dtype=torch.bfloat16))

    def forward(self, hidden):
        return cce.linear(hidden.bfloat16(), self.weight, self.bias, activation="gelu", out_dtype=torch.float32)


class GatedBlock(torch.nn.Module):
    """x + W_down (silu(W_gate n) * (W_up n)), n the RMS norm of x, in a 32-bit residual stream."""

    def __init__(self, dim, inner=None, device="cuda"):
        super().__init__()
        inner = 4 * dim if inner is None else inner

        def weight(n, k):
            return torch.nn.Parameter((torch.randn(n, k, device=device) / k ** 0.5).bfloat16())
        self.norm = torch.nn.Parameter(torch.ones(dim, device=device))
        self.gate, self.up, self.down = weight(inner, dim), weight(inner, dim), weight(dim, inner)

    def forward(self, hidden):
        n = cce.rms_norm(hidden, self.norm, out_dtype=torch.bfloat16)
        return cce.linear(cce.gated_linear(n, self.gate, self.up), self.down, residual=hidden, out_dtype=torch.float32)


BLOCKS = {"none": None, "transform": Transform, "gated": GatedBlock}


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


def train(norm="layer", steps=20, tokens=1024, dim=128, vocab=4096, lr=0.5, max_norm=1.0, seed=0, block="none",
          optimizer="sgd"):
    """The losses and the gradient norms of the steps."""
    torch.manual_seed(seed)
    head = Head(dim, vocab, norm)
    front = BLOCKS[block](dim) if BLOCKS[block] else None
    parameters = list(head.parameters()) + (list(front.parameters()) if front else [])
    if optimizer != "sgd":
        # (a learning rate of 0.5 is for plain gradients)
        opt = cce.AdamW(parameters, lr=lr * 1e-2, state_bits=8 if optimizer == "adamw8" else 32, master_weights=True)
    hidden = torch.randn(4, tokens // 4, dim, device="cuda") * 3 + 0.5
    targets = torch.randint(0, vocab, (4, tokens // 4), device="cuda")
    # every position predicts the next one: the last of each sequence has no target
    hidden, targets = hidden[:, :-1], targets[:, 1:]
    losses, norms = [], []
    for _ in range(steps):
        loss = head(front(hidden) if front else hidden, targets)
        for p in parameters:
            p.grad = None
        loss.backward()
        if optimizer == "sgd":
            norms.append(cce.clip_grad_norm_(parameters, max_norm))
            with torch.no_grad():
                for p in parameters:
                    p.sub_(p.grad, alpha=lr)
        else:
            norms.append(cce.cce_grad_norm([p.grad for p in parameters]))
            opt.step(grad_norm=norms[-1], max_norm=max_norm)
        losses.append(loss.detach())
    cce.raise_pending_errors()
    return [float(v) for v in losses], [float(v) for v in norms]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--norm", choices=("layer", "rms"), default="layer")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--block", choices=tuple(BLOCKS), default="none")
    ap.add_argument("--optimizer", choices=("sgd", "adamw", "adamw8"), default="sgd")
    a = ap.parse_args()
    for i, (loss, norm) in enumerate(zip(*train(a.norm, a.steps, a.tokens, block=a.block, optimizer=a.optimizer))):
        print(f"step {i:3d}  loss {loss:.4f}  gradient norm {norm:.4f}")


if __name__ == "__main__":
    main()
