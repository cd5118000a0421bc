"""float64 reference of the root-mean-square norm, written from its definition
in include/mok.h (test infrastructure; no code shared with the HIP path)."""
from __future__ import annotations

import numpy as np

from .moe_oracle import bf16_round


def norm_forward(x, weight, residual=None, eps=1e-6):
    """(y, z, rstd): z is the stream as it is stored, in bf16."""
    # (fp32 addition first, as two bf16 values are added: its own rounding can only matter at a tie)
    z = x if residual is None else bf16_round((x.astype(np.float32) + residual.astype(np.float32)).astype(np.float64))
    rstd = 1.0 / np.sqrt((z * z).mean(1) + eps)
    y = z * rstd[:, None]
    return (y if weight is None else y * weight), z, rstd


def norm_backward(dy, z, rstd, weight, d_sum=None):
    """(dx, dw) with rstd = rstd(z)."""
    xh = z * rstd[:, None]
    g = dy if weight is None else dy * weight
    dx = rstd[:, None] * (g - xh * (g * xh).mean(1, keepdims=True))
    return (dx if d_sum is None else dx + d_sum), (dy * xh).sum(0)
