"""Embedding lookup with scaling and its gradient, in fp64.

TEST INFRASTRUCTURE ONLY (see the package header).

The definition: out[t] = scale * table[ids[t]], zeros for an id outside [0, V);
d_table[v] = scale * sum over t with ids[t] = v of d_out[t].

Pins (tests/test_oracle_tokens.py): hand-computed rows, a one-hot product, and
torch.autograd in fp64 over the definition.
"""
from __future__ import annotations

import numpy as np


def forward(ids, table, scale=1.0):
    table = np.asarray(table, dtype=np.float64)
    ids = np.asarray(ids)
    out = np.zeros((ids.size, table.shape[1]))
    for t, i in enumerate(ids.ravel()):
        if 0 <= i < table.shape[0]:
            out[t] = scale * table[i]
    return out


def backward(d_out, ids, V, scale=1.0):
    """(d_table [V, d], the sum of magnitudes behind each entry, tokens per row)"""
    d_out = np.asarray(d_out, dtype=np.float64)
    ids = np.asarray(ids).ravel()
    total, mags = np.zeros((V, d_out.shape[1])), np.zeros((V, d_out.shape[1]))
    n = np.zeros(V, dtype=np.int64)
    for t, i in enumerate(ids):
        if 0 <= i < V:
            total[i] += d_out[t]
            mags[i] += np.abs(d_out[t])
            n[i] += 1
    return scale * total, abs(scale) * mags, n
