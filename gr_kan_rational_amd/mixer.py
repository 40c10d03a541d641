"""The channel mixer of a GR-KAN transformer block on the block operators:

    y = x + F2(F1(norm(x)) W1^T + b1) W2^T + b2

F1 is applied where the norm's result is formed, F2 in the epilogue of the first product, the residual in
that of the second: three launches forward, no tensor of [rows, hidden] but F2's result and, for training,
the product before it.  The pages start a GR-KAN layer's first activation as the identity and its second as a
Swish ("FlashKAT ...", Paper-Notes page, section "损失函数 / 训练策略"); the Swish coefficients below are this
library's own least-squares fit.
"""
from __future__ import annotations

import math

import torch

from .block import GRKANGroupNorm, GRKANLinearAct

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
