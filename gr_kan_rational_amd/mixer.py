"""The channel mixer of a GR-KAN transformer block on the block operators, and a deep stack of them.  The mixer:

    y = x + F2(F1(norm(x)) W1^T + b1) W2^T + b2

F1 is applied where the norm's result is formed, F2 in the epilogue of the first product, the residual in
that of the second: three launches forward, no tensor of [rows, hidden] but F2's result and, for training,
the product before it.  The pages start a GR-KAN layer's first activation as the identity and its second as a
Swish ("FlashKAT ...", Paper-Notes page, section "损失函数 / 训练策略"); the Swish coefficients below are this
library's own least-squares fit.

The stack: what passes from one mixer to the next, with a residual scale, stochastic depth and the norms on either
side, is one operator, and the products may run in 8 bits.
"""
from __future__ import annotations

import math

import torch

from .binding import GRKANFunction
from .block import GRKANGroupNorm, GRKANLinearAct
from .train import GRKANFp8Linear, GRKANResidualNorm

# x / (1 + e^-x) on [-5, 5] by degrees (5, 4) with an even, positive denominator: within 7e-5.
SWISH_A = (0.0, 0.5, 0.249944, 0.0526866, 0.00555034, 0.000244433)
SWISH_B = (0.0, 0.105373, 0.0, 0.000488866)
IDENTITY_A = (0.0, 1.0, 0.0, 0.0, 0.0, 0.0)
IDENTITY_B = (0.0, 0.0, 0.0, 0.0)


class GRKANMixer(torch.nn.Module):
    """``forward(x)`` for bfloat16 x [..., dim] or [samples, ..., dim].

    ``norm_groups`` = 0 is the norm per token; otherwise x is [samples, positions, dim] and the channels
    are normalised in that many groups over the positions.  Weights are bfloat16; biases, the norm's
    parameters and the coefficients float32."""

    def __init__(self, dim: int, hidden: int, n_groups: int = 8, norm_groups: int = 0, device=None):
        super().__init__()
        if dim % n_groups or hidden % n_groups:
            raise ValueError("dim and hidden must be multiples of n_groups")
        self.n_groups, self.norm_groups = n_groups, norm_groups

        def coefficients(values):
            return torch.nn.Parameter(torch.tensor(values, device=device).repeat(n_groups, 1))

        def weight(rows, cols):
            w = torch.randn(rows, cols, device=device) / math.sqrt(cols)
            return torch.nn.Parameter(w.to(torch.bfloat16))

        self.norm_weight = torch.nn.Parameter(torch.ones(dim, device=device))
        self.norm_bias = torch.nn.Parameter(torch.zeros(dim, device=device))
        self.A1, self.B1 = coefficients(IDENTITY_A), coefficients(IDENTITY_B)
        self.A2, self.B2 = coefficients(SWISH_A), coefficients(SWISH_B)
        self.W1, self.b1 = weight(hidden, dim), torch.nn.Parameter(torch.zeros(hidden, device=device))
        self.W2, self.b2 = weight(dim, hidden), torch.nn.Parameter(torch.zeros(dim, device=device))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        rows = x if self.norm_groups else x.reshape(-1, x.shape[-1])
        h = GRKANGroupNorm.apply(rows, self.norm_groups or 1, self.norm_weight, self.norm_bias, 1e-5, "rational",
                                 self.A1, self.B1, self.n_groups)
        h = GRKANLinearAct.apply(h, self.W1, self.b1, "rational", self.A2, self.B2, self.n_groups)
        y = GRKANLinearAct.apply(h, self.W2, self.b2, "none", None, None, self.n_groups, rows)
        return y.view(x.shape)


class GRKANStack(torch.nn.Module):
    """``depth`` channel mixers one after another and a last norm: for each,

        f = F2(F1(z) W1^T + b1) W2^T + b2,    h = h + scale gate post(f),    z = norm(h)

    and z of the last one is the result.  ``forward(x)`` takes bfloat16 x [..., dim], samples first (of x [dim]
    one).  ``products``
    is "bf16" or "fp8" (e4m3, a scale for each block of 128; ``sums`` "fp32" or "fast" as ``grkan_fp8_matmul``'s).  ``post`` is "none", "layer" or "rms".  ``scale``
    is the residual scale's first value.  ``drop`` is the rate at which, in training, a sample's branch is left
    out (the others scaled up to match), rising from 0 at the first mixer.  Weights are bfloat16, all else
    float32."""

    def __init__(self, depth: int, dim: int, hidden: int, n_groups: int = 8, products: str = "bf16", post: str = "none",
                 scale: float = 0.1, drop: float = 0.0, device=None, sums: str = "fp32"):
        super().__init__()
        if dim % n_groups or hidden % n_groups:
            raise ValueError("dim and hidden must be multiples of n_groups")
        if products not in ("bf16", "fp8"):
            raise ValueError('products must be "bf16" or "fp8"')
        if sums not in ("fp32", "fast"):
            raise ValueError('sums must be "fp32" or "fast"')
        if not 0.0 <= drop < 1.0:
            raise ValueError("drop must be in [0, 1)")
        self.n_groups, self.products, self.post, self.drop, self.sums = n_groups, products, post, drop, sums

        def vector(value, size):
            return torch.nn.Parameter(torch.full((size,), value, device=device))

        def coefficients(values):
            return torch.nn.Parameter(torch.tensor(values, device=device).repeat(n_groups, 1))

        def weight(rows, cols):
            w = torch.randn(rows, cols, device=device) / math.sqrt(cols)
            return torch.nn.Parameter(w.to(torch.bfloat16))

        self.blocks = torch.nn.ModuleList()
        for _ in range(depth):
            m = torch.nn.ParameterDict({
                "A1": coefficients(IDENTITY_A), "B1": coefficients(IDENTITY_B), "A2": coefficients(SWISH_A),
                "B2": coefficients(SWISH_B), "W1": weight(hidden, dim), "b1": vector(0.0, hidden),
                "W2": weight(dim, hidden), "b2": vector(0.0, dim), "scale": vector(scale, dim),
                "norm_weight": vector(1.0, dim), "norm_bias": vector(0.0, dim)})
            if post != "none":
                m["post_weight"] = vector(1.0, dim)
            if post == "layer":
                m["post_bias"] = vector(0.0, dim)
            self.blocks.append(m)
        self.norm_weight, self.norm_bias = vector(1.0, dim), vector(0.0, dim)

    def branch(self, m, z: torch.Tensor) -> torch.Tensor:
        """f of one mixer."""
        if self.products == "fp8":
            y = GRKANFp8Linear.apply(z, m["W1"], m["b1"], "rational", m["A1"], m["B1"], self.n_groups, self.sums)
            return GRKANFp8Linear.apply(y, m["W2"], m["b2"], "rational", m["A2"], m["B2"], self.n_groups, self.sums)
        y = GRKANFunction.apply(z, m["A1"], m["B1"], self.n_groups)
        y = GRKANLinearAct.apply(y, m["W1"], m["b1"], "rational", m["A2"], m["B2"], self.n_groups)
        return GRKANLinearAct.apply(y, m["W2"], m["b2"])

    def gates(self, x: torch.Tensor):
        """Each mixer's gate of the samples, or None: 1 / (1 - rate) for those that are kept, else 0."""
        if not self.training or self.drop == 0.0 or not len(self.blocks):
            return [None] * len(self.blocks)
        depth = len(self.blocks)
        rates = torch.arange(depth, device=x.device, dtype=torch.float32).mul_(self.drop / max(depth - 1, 1))
        samples = (x.shape[0], *(1,) * (x.dim() - 1)) if x.dim() > 1 else (1,)
        kept = torch.rand(depth, samples[0], device=x.device) >= rates[:, None]
        return list((kept / (1.0 - rates)[:, None]).view(depth, *samples))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        x = x.contiguous()
        # mixer k normalises with its own vectors, so the norm after mixer k is mixer k + 1's
        norms = [(m["norm_weight"], m["norm_bias"]) for m in self.blocks] + [(self.norm_weight, self.norm_bias)]
        h = x
        z = GRKANGroupNorm.apply(x.view(-1, x.shape[-1]), 1, *norms[0], 1e-5).view(x.shape)
        for m, gate, (w, b) in zip(self.blocks, self.gates(x), norms[1:]):
            f = self.branch(m, z)
            h, z = GRKANResidualNorm.apply(h, f, "layer", w, b, m["scale"], gate, self.post,
                                           m["post_weight"] if self.post != "none" else None,
                                           m["post_bias"] if self.post == "layer" else None)
        return z
