"""Trains a deep stack of GR-KAN channel mixers to imitate another on random tokens (one GPU): products in 8 bits,
AdamW with 8-bit states over all tensors at once, the gradients scaled down to a greatest norm.

    python examples/train_stack.py [--steps 60] [--samples 32] [--positions 64] [--depth 4] [--dim 192]
                                   [--hidden 768] [--products fp8] [--bits 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gr_kan_rational_amd import GRKANAdamW  # noqa: E402
from gr_kan_rational_amd.mixer import GRKANStack  # noqa: E402


def train(steps: int, samples: int, positions: int, depth: int, dim: int, hidden: int, products: str = "fp8", bits: int = 8,
          seed: int = 0, quiet: bool = False) -> list[float]:
    torch.manual_seed(seed)
    teacher = GRKANStack(depth, dim, hidden, device="cuda").requires_grad_(False).eval()
    student = GRKANStack(depth, dim, hidden, products=products, drop=0.05, device="cuda")
    matrices = [p for p in student.parameters() if p.dtype == torch.bfloat16]
    vectors = [p for p in student.parameters() if p.dtype != torch.bfloat16]
    opt = GRKANAdamW([{"params": matrices, "weight_decay": 0.05}, {"params": vectors, "weight_decay": 0.0}], lr=2e-3,
                     bits=bits)
    losses = []
    for step in range(steps):
        x = torch.randn(samples, positions, dim, device="cuda").to(torch.bfloat16)
        loss = (student(x).float() - teacher(x).float()).square().mean()
        opt.zero_grad(set_to_none=True)
        loss.backward()
        norm = torch.stack([p.grad.float().norm() for p in student.parameters()]).norm()
        opt.step(grad_scale=(1.0 / norm).clamp_max(1.0))
        losses.append(float(loss.detach()))
        if not quiet and step % 10 == 0:
            print(f"step {step:4d}  loss {losses[-1]:.4f}", flush=True)
    return losses


def main():
    p = argparse.ArgumentParser()
    for name, value in (("steps", 60), ("samples", 32), ("positions", 64), ("depth", 4), ("dim", 192), ("hidden", 768),
                        ("bits", 8)):
        p.add_argument(f"--{name}", type=int, default=value)
    p.add_argument("--products", default="fp8")
    a = p.parse_args()
    losses = train(a.steps, a.samples, a.positions, a.depth, a.dim, a.hidden, a.products, a.bits)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
