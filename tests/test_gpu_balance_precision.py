"""The balance loss and its gradient keep fp32 precision wherever the logits lie.

Tolerances, in units of u = 2^-24.  An affinity takes the hardware's exponential
and root (2u each), the product that carries the exponent's low part (u), the
polynomial (u, halved by the root) and their product (u): 7u.  A row's sum adds
7u of its terms and 10u of additions, its inverse and the product with it 2u, the
mean of one token 2u: 28u at worst, compared to 32u.  The roundings are
independent, an rms of 0.6 of each bound: below 3u in the affinity and 4u with the
row's, compared to 6u.  A gradient element adds the reciprocal (2u) and four
products, relative to the two terms of its difference: 40u and 8u."""
import numpy as np
import pytest
import torch

import moe_expert_routing_sqrt_amd as M
from oracle import balance_loss as OL

from gpu_util import dev_f32, dev_i32, host, need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _rms(x):
    return float(np.sqrt(np.mean(np.square(x))))


# T, E, sequences, counted tokens of a sequence (0: all): one launch, short sequences, long ones
FORMS = [(40, 64, 40, 0), (30, 37, 30, 0), (200, 64, 200, 0), (150, 41, 150, 0), (400, 256, 4, 1), (200, 600, 2, 1),
         (300, 1000, 3, 1)]


@pytest.mark.parametrize("centre", [-165.0, -70.0, -12.0, 0.0, 30.0])
@pytest.mark.parametrize("T,E,n,counted", FORMS)
def test_probabilities_and_gradient_at_any_logit(T, E, n, counted, centre):
    """One token a sequence, so that its mean hides nothing."""
    dev = need_gpu()
    print(f"balance loss T={T} E={E} n={n} around {centre}", flush=True)
    rng = np.random.default_rng(T + E)
    L = (centre + 1.5 * rng.normal(size=(T, E))).astype(np.float32)
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :2].astype(np.int32)
    off = (np.arange(n + 1) * T // n).astype(np.int32)
    mask = None
    if counted:
        mask = np.zeros(T, dtype=bool)
        mask[off[:-1] + 5] = True
    sh, Ld = M.shape(T, 1, E, 1, 1, 2, 1, 1), dev_f32(L, dev)
    kw = dict(seq_offsets=dev_i32(off, dev), token_mask=None if mask is None else torch.from_numpy(mask).to(dev))
    loss, counts, prob, dprob = M.balance_loss(sh, Ld, dev_i32(idx, dev), 1.0, **kw)
    dl = M.balance_loss_backward(sh, Ld, dprob, **kw)
    torch.cuda.synchronize()
    ref = OL.forward(L, idx, 1.0, off, mask)
    rel = (host(prob) - ref[2]) / ref[2]
    assert np.abs(rel).max() <= 32 * U, np.abs(rel).max() / U
    assert _rms(rel) <= 6 * U, _rms(rel) / U
    # each sequence's loss has few terms of 32u; the sum over sequences adds in
    # fp32 by trees and chains of at most 32
    assert abs(float(loss) - ref[0]) <= (32 + 64) * U * ref[0]
    dp = host(dprob).astype(np.float64)
    rl = OL.backward(L, dp, off, mask)
    on = np.arange(T) if mask is None else np.flatnonzero(mask)
    seq = np.searchsorted(off, on, side="right") - 1
    a = OL.affinity(L[on])
    S = a.sum(1, keepdims=True)
    e = np.exp(-np.abs(L[on].astype(np.float64)))
    sig = np.where(L[on] >= 0, 1 / (1 + e), e / (1 + e))
    terms = (dp[seq] + (dp[seq] * a).sum(1, keepdims=True) / S) / S * sig / (2 * a)
    rel = (host(dl)[on] - rl[on]) / terms
    assert np.abs(rel).max() <= 40 * U, np.abs(rel).max() / U
    assert _rms(rel) <= 8 * U, _rms(rel) / U


def test_infinitely_negative_logits_are_experts_without_a_share():
    dev = need_gpu()
    for T, E, n in ((20, 64, 2), (300, 64, 30), (300, 64, 2), (100, 600, 1)):
        rng = np.random.default_rng(E)
        L = rng.normal(size=(T, E)).astype(np.float32)
        L[:, 3::4] = -np.inf
        L[7] = -np.inf                                         # nothing left of this row
        idx = np.tile(np.array([0, 1], dtype=np.int32), (T, 1))
        off = (np.arange(n + 1) * T // n).astype(np.int32)
        sh, Ld, kw = M.shape(T, 1, E, 1, 1, 2, 1, 1), dev_f32(L, dev), dict(seq_offsets=dev_i32(off, dev))
        loss, _, prob, dprob = M.balance_loss(sh, Ld, dev_i32(idx, dev), 1.0, **kw)
        dl = host(M.balance_loss_backward(sh, Ld, dprob, **kw))
        torch.cuda.synchronize()
        ref = OL.forward(L, idx, 1.0, off)
        assert not prob[:, 3::4].any() and np.abs(host(prob) - ref[2]).max() <= 1e-5 * ref[2].max()
        assert abs(float(loss) - ref[0]) <= 1e-5 * ref[0]
        assert np.isfinite(dl).all() and not dl[7].any() and not dl[:, 3::4].any()


def test_rows_near_and_past_the_last_affinity():
    """Below a logit of -174 an affinity has no fp32 value: such rows vanish or hold
    probabilities, and nothing is infinite or NaN."""
    dev = need_gpu()
    for T, E, n in ((20, 64, 2), (300, 64, 30), (300, 64, 2), (100, 600, 1)):
        L = np.linspace(-172, -215, T).astype(np.float32)[:, None] + np.zeros((1, E), np.float32)
        idx = np.tile(np.array([0, 1], dtype=np.int32), (T, 1))
        off = (np.arange(n + 1) * T // n).astype(np.int32)
        sh, Ld, kw = M.shape(T, 1, E, 1, 1, 2, 1, 1), dev_f32(L, dev), dict(seq_offsets=dev_i32(off, dev))
        loss, _, prob, dprob = M.balance_loss(sh, Ld, dev_i32(idx, dev), 1.0, **kw)
        dl = host(M.balance_loss_backward(sh, Ld, dprob, **kw))
        torch.cuda.synchronize()
        assert np.isfinite(dl).all() and bool(torch.isfinite(prob).all()) and bool(torch.isfinite(loss).all())
        assert float(prob.sum(1).max()) <= 1 + 1e-5
