"""Layer and RMS norm of rows, forward and backward, in float64.

Test infrastructure only (see the package header).
    xh = (x - mean) rstd, y = xh w + b;  RMS: mean = 0
    dx = rstd (w dy - mean(w dy) - xh mean(w dy xh))   (RMS: without the middle term)
    dw = sum over rows of dy xh,  db = sum over rows of dy

Pins: tests/test_oracle_around.py (central differences, torch autograd)."""

from __future__ import annotations

import numpy as np


def statistics(x, kind: str, eps: float):
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1) if kind == "layer" else np.zeros(x.shape[0])
    return mean, 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)


def forward(x, weight, bias, kind: str, eps: float):
    """(y, mean, rstd); weight and bias may be None."""
    mean, rstd = statistics(x, kind, eps)
    y = (np.asarray(x, dtype=np.float64) - mean[:, None]) * rstd[:, None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def backward(grad_y, x, mean, rstd, weight, kind: str):
    """(dx, dw, db)."""
    gy = np.asarray(grad_y, dtype=np.float64)
    xh = (np.asarray(x, dtype=np.float64) - mean[:, None]) * rstd[:, None]
    g = gy if weight is None else gy * weight
    dx = g - xh * (g * xh).mean(axis=1, keepdims=True)
    if kind == "layer":
        dx = dx - g.mean(axis=1, keepdims=True)
    return dx * rstd[:, None], (gy * xh).sum(axis=0), gy.sum(axis=0)
