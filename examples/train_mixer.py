"""Trains one GR-KAN channel mixer to imitate another on random tokens (one GPU).

    python examples/train_mixer.py [--steps 60] [--tokens 4096] [--dim 192] [--hidden 768]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gr_kan_rational_amd.mixer import GRKANMixer  # noqa: E402


def train(steps: int, tokens: int, dim: int, hidden: int, seed: int = 0, quiet: bool = False) -> list[float]:
    torch.manual_seed(seed)
    teacher = GRKANMixer(dim, hidden, device="cuda").requires_grad_(False)
    student = GRKANMixer(dim, hidden, device="cuda")
    opt = torch.optim.AdamW(student.parameters(), lr=2e-3, weight_decay=0.0)
    losses = []
    for step in range(steps):
        x = torch.randn(tokens, dim, device="cuda").to(torch.bfloat16)
        loss = (student(x).float() - teacher(x).float()).square().mean()
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
        if not quiet and step % 10 == 0:
            print(f"step {step:4d}  loss {losses[-1]:.4f}", flush=True)
    return losses


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--dim", type=int, default=192)
    p.add_argument("--hidden", type=int, default=768)
    a = p.parse_args()
    losses = train(a.steps, a.tokens, a.dim, a.hidden)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
