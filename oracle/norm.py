"""Layer norm with the residual add, and its backward, in fp64.

TEST INFRASTRUCTURE ONLY (see the package header).

The definition: s = x + r (rounded to the stored type by the caller's inputs),
mu = sum(s)/d, rstd = 1/sqrt(sum((s - mu)^2)/d + eps), y = (s - mu) rstd w + b.
Backward for dy, with xh = (s - mu) rstd and q = dy w:
    dx = rstd (q - mean(q) - xh mean(q xh)) + d_sum
    dw = sum_t dy xh,   db = sum_t dy

Pins (tests/test_oracle_training.py): a hand-computed row, torch.autograd in
fp64 over the forward's definition, and central differences.
"""
from __future__ import annotations

import numpy as np


def forward(s, w, b=None, eps=1e-5):
    """(y, mean, rstd) of rows s [rows, d]."""
    s = np.asarray(s, dtype=np.float64)
    d = s.shape[1]
    mean = s.sum(1) / d
    c = s - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).sum(1) / d + eps)
    y = c * rstd[:, None] * np.asarray(w, dtype=np.float64)
    if b is not None:
        y = y + np.asarray(b, dtype=np.float64)
    return y, mean, rstd


def backward(dy, s, w, mean, rstd, d_sum=None):
    """(dx, dw, db) from the forward's statistics."""
    dy, s, w = (np.asarray(a, dtype=np.float64) for a in (dy, s, w))
    mean, rstd = (np.asarray(a, dtype=np.float64)[:, None] for a in (mean, rstd))
    d = s.shape[1]
    xh = (s - mean) * rstd
    q = dy * w
    dx = rstd * (q - q.sum(1, keepdims=True) / d - xh * ((q * xh).sum(1, keepdims=True) / d))
    if d_sum is not None:
        dx = dx + np.asarray(d_sum, dtype=np.float64)
    return dx, (dy * xh).sum(0), dy.sum(0)
