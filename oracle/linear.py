"""Oracle of the product with one 4-bit matrix (float64): y = act(x w^T) + residual, w dequantised from
the stored codes and scales; SwiGLU takes rows 0..N/2-1 as gate and the others as up."""
from __future__ import annotations

import numpy as np


def silu(v):
    return v * (0.5 * (1.0 + np.tanh(0.5 * v)))


def linear(x, w, swiglu: bool = False, residual=None):
    """x [T][K], w [N][K] float64 -> [T][N] or [T][N/2]."""
    y = x @ w.T
    if swiglu:
        half = w.shape[0] // 2
        y = silu(y[:, :half]) * y[:, half:]
    return y if residual is None else y + residual
