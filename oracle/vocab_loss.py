"""Losses on logits over a vocabulary and their gradients, in fp64: distillation
from a teacher's top logits, and the clipped policy loss with a KL term.

TEST INFRASTRUCTURE ONLY (see the package header).

The definitions, for a row x of V logits at temperature tau with q =
softmax(x / tau):
  distill  p = softmax(t / tau) over the entries with an index in [0, V) and a
           logit above -inf;  l = tau^2 sum_j p_j (log p_j - log q[i_j]);
           dl/dx = tau (q - sum_j p_j e_{i_j})
  policy   logp = log q[token], r = exp(logp - old), d = ref - logp;
           l = -min(r A, clamp(r, 1 - lo, 1 + hi) A) + kl (exp(d) - d - 1);
           dl/dlogp = -[r A <= clamp(r) A] r A + kl (1 - exp(d));
           dl/dx = dl/dlogp / tau (e_token - q)
Rows of weight 0, without an entry, or with a token outside [0, V) count nothing.

Pins (tests/test_oracle_tokens.py): closed forms for two logits, a pure-Python
brute force, torch.autograd in fp64 and central differences.
"""
from __future__ import annotations

import numpy as np


def softmax_row(x, tau):
    """(q, log q, max, sum of exp((x - max)/tau)) of one row"""
    x = np.asarray(x, dtype=np.float64)
    m = x.max()
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        z = (x - m) / tau
        e = np.exp(z)
        s = e.sum()
        return e / s, z - np.log(s), m, s


def _weights(T, weight):
    return np.full(T, 1.0 / T) if weight is None else np.asarray(weight, dtype=np.float64)


def teacher_row(idx, t, V, tau):
    """(valid entries' positions in the row's list, their probabilities and log-probabilities)"""
    t = np.asarray(t, dtype=np.float64)
    ok = np.flatnonzero((idx >= 0) & (idx < V) & (t != -np.inf))
    if len(ok) == 0:
        return ok, t[ok], t[ok]
    z = (t[ok] - t[ok].max()) / tau
    s = np.exp(z).sum()
    return ok, np.exp(z) / s, z - np.log(s)


def distill(x, idx, t, tau=1.0, weight=None, grad=1.0):
    """dict of loss, row_loss [T], stats [T, 2] and dlogits [T, V]"""
    x = np.asarray(x, dtype=np.float64)
    T, V = x.shape
    w = _weights(T, weight)
    row, stats, dx = np.zeros(T), np.zeros((T, 2)), np.zeros((T, V))
    for r in range(T):
        ok, p, logp = teacher_row(idx[r], t[r], V, tau)
        if w[r] == 0 or len(ok) == 0:
            continue
        q, logq, m, s = softmax_row(x[r], tau)
        at = np.asarray(idx[r])[ok]
        some = p > 0
        row[r] = tau * tau * (p[some] * (logp[some] - logq[at[some]])).sum()
        stats[r] = m, s
        d = q.copy()
        np.subtract.at(d, at, p)
        dx[r] = grad * w[r] * tau * d
    live = w != 0
    return dict(loss=(w[live] * row[live]).sum(), row_loss=row, stats=stats, dlogits=dx)


def policy(x, tok, old, adv, ref=None, clip=(0.2, 0.2), kl=0.0, tau=1.0, weight=None, grad=1.0):
    """dict of loss, row_loss, logp [T], stats [T, 2] and dlogits [T, V]"""
    x = np.asarray(x, dtype=np.float64)
    T, V = x.shape
    w = _weights(T, weight)
    row, lp, stats, dx = np.zeros(T), np.zeros(T), np.zeros((T, 2)), np.zeros((T, V))
    for r in range(T):
        if w[r] == 0 or not 0 <= tok[r] < V:
            continue
        q, logq, m, s = softmax_row(x[r], tau)
        logp = logq[tok[r]]
        ratio, a = np.exp(logp - float(old[r])), float(adv[r])
        free, cut = ratio * a, min(max(ratio, 1 - clip[0]), 1 + clip[1]) * a
        if a == 0 and ratio == np.inf:  # an advantage of 0 counts 0 beside any ratio
            free = 0.0
        row[r] = -min(free, cut)
        slope = -free if free <= cut else 0.0
        if kl:
            d = float(ref[r]) - logp
            row[r] += kl * (np.expm1(d) - d)
            slope -= kl * np.expm1(d)
        lp[r] = logp
        stats[r] = m, s
        d = -q
        d[tok[r]] += 1
        dx[r] = grad * w[r] * slope / tau * d
    live = w != 0
    return dict(loss=(w[live] * row[live]).sum(), row_loss=row, logp=lp, stats=stats, dlogits=dx)
