"""The router's balance loss, its per-expert counts and its gradient, in fp64.

TEST INFRASTRUCTURE ONLY (see the package header).

p[t,e] = a[t,e] / sum_e a[t,e], a = sqrt(softplus(l)) (0 for a row whose
affinities all vanish); for sequence s with T_s counted tokens:
    c[s,e] = slots of counted tokens on e,  f = E c / (k T_s),  P = sum_t p / T_s
    loss = alpha / n * sum_s sum_e f P
    dprob[s,e] = alpha f / (n T_s)
Gradient with c fixed: dl[t,e] = g (dprob_e - sum_j dprob_j p_j) / S * sig(l) / (2 a).

A loop over tokens, one at a time; a sequence without a counted token adds 0.

Pins (tests/test_oracle_training.py): a uniform router (loss = alpha), a
collapsed router, counts by hand, torch.autograd in fp64 and central
differences.
"""
from __future__ import annotations

import numpy as np


def affinity(l):
    l = np.asarray(l, dtype=np.float64)
    return np.sqrt(np.logaddexp(0.0, l))


def forward(logits, idx, alpha, offsets=None, mask=None):
    """(loss, counts [n, E], prob [n, E], dprob [n, E])."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    k = idx.shape[1]
    off = [0, T] if offsets is None else [int(o) for o in offsets]
    n = len(off) - 1
    counts = np.zeros((n, E), dtype=np.int64)
    prob = np.zeros((n, E))
    dprob = np.zeros((n, E))
    loss = 0.0
    for s in range(n):
        tokens = [t for t in range(off[s], off[s + 1]) if mask is None or mask[t]]
        if not tokens:
            continue
        for t in tokens:
            a = affinity(logits[t])
            if a.sum() != 0:  # NaN too: such a row has probabilities, and they are NaN
                prob[s] += a / a.sum()
            for e in idx[t]:
                if 0 <= e < E:
                    counts[s, e] += 1
        prob[s] /= len(tokens)
        f = E * counts[s] / (k * len(tokens))
        loss += alpha / n * float((f * prob[s]).sum())
        dprob[s] = alpha * f / (n * len(tokens))
    return loss, counts, prob, dprob


def backward(logits, dprob, offsets=None, mask=None, grad_loss=1.0, d_extra=None):
    logits = np.asarray(logits, dtype=np.float64)
    dprob = np.asarray(dprob, dtype=np.float64)
    T, E = logits.shape
    off = [0, T] if offsets is None else [int(o) for o in offsets]
    out = np.zeros((T, E)) if d_extra is None else np.array(d_extra, dtype=np.float64)
    for s in range(len(off) - 1):
        for t in range(off[s], off[s + 1]):
            if mask is not None and not mask[t]:
                continue
            l = logits[t]
            a = affinity(l)
            S = a.sum()
            if S == 0:
                continue
            da = grad_loss * (dprob[s] - (dprob[s] * a).sum() / S) / S
            with np.errstate(over="ignore"):
                sig = np.where(l >= 0, 1.0 / (1.0 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1.0 + np.exp(-np.abs(l))))
            out[t] += np.where(a != 0, da * sig / (2.0 * np.where(a != 0, a, 1.0)), 0.0)
    return out
