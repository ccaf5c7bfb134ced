"""GPU parity of the policy loss where the ratio or the KL term is far from 1:
differences of log-probabilities that fp32's exponential does not hold, infinite
ones, and advantages of 0 beside them.

Expected values are formed here in fp64.  A ratio of 0 advantage counts 0 however
large it is; a loss beyond fp32 is infinite; a gradient's factor beyond fp32 is its
largest number, so that entries of probability 0 keep a gradient of 0.

Tolerances (U = 2^-24).  S: the relative error of a row's sum of exponentials, as
in test_gpu_vocab_loss.py (46 U + 6 U mean |z| + 4 U here, one piece a thread).  The
ratio's relative error is logp's absolute one, S + 4 U, and 8 U of its exponential
and products; the gradient's q adds U (3 |z| + 8) + S; each store half a step."""
import numpy as np
import pytest
import torch

import moe_expert_routing_sqrt_amd as M

from gpu_util import host, need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
MAX = float(np.finfo(np.float32).max)
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": U, "bf16": 2.0 ** -8}
DIFF = [-200.0, -105.0, -80.0, 80.0, 88.5, 89.0, 91.3, 95.0, 97.7, 100.0, 103.0, 105.0, 200.0, 600.0, float("inf")]
CLIP = (0.2, 0.28)


def _rows(V, T, xt, dev):
    g = torch.Generator(device=dev).manual_seed(V)
    x = 2 * torch.randn(T, V, generator=g, device=dev)
    x[:, V - V // 10:] = float("-inf")
    x = x.to(DT[xt])
    tok = torch.randint(0, V - V // 10, (T,), generator=g, device=dev, dtype=torch.int32)
    h = host(x).astype(np.float64)
    z = h - h.max(1, keepdims=True)
    e = np.exp(z)
    s = e.sum(1, keepdims=True)
    zz = np.where(e > 0, np.abs(z), 0.0)
    S = U * (50 + V / 1024 + 6 * (e * zz).sum(1) / s[:, 0])
    logp = z[np.arange(T), host(tok)] - np.log(s[:, 0])
    return x, tok, logp, e / s, zz, S


def _grad(slope, w, q, tok):
    """w slope ([token] - q), the factor held to fp32's range"""
    k = np.clip(np.clip(slope, -1e300, 1e300) * w, -MAX, MAX)[:, None]
    return k * ((np.arange(q.shape[1]) == tok[:, None]) - q)


def _check(got, row, row_tol, dx, dx_rel, dt):
    have = host(got[1]).astype(np.float64)
    big = np.abs(row) > MAX
    assert (have[big] == np.sign(row[big]) * np.inf).all()
    near = ~big & (np.abs(row) < 0.99 * MAX)
    assert (np.abs(have[near] - row[near]) <= row_tol[near] + U * np.abs(row[near]) + 1e-44).all()
    d = host(got[4]).astype(np.float64)
    assert not np.isnan(d).any()
    fits = np.abs(dx) < 0.99 * MAX
    tol = np.abs(dx) * (dx_rel + HALF[dt]) + 1e-38
    assert (np.abs(d[fits] - dx[fits]) <= tol[fits]).all()
    assert (d[dx == 0] == 0).all()


@pytest.mark.parametrize("V", [300, 9000, 70001])
@pytest.mark.parametrize("xt,dt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_large_ratios(V, xt, dt):
    dev = need_gpu()
    A = [1.0, 1.7, 0.0, -0.0, -1.0, -1e-30]
    T = len(DIFF) * len(A)
    x, tok, logp, q, zz, S = _rows(V, T, xt, dev)
    diff = np.repeat(DIFF, len(A))
    adv = torch.tensor(A, device=dev).repeat(len(DIFF))
    old = torch.from_numpy((logp - diff).astype(np.float32)).to(dev)
    w = torch.full((T,), 0.25, device=dev)
    with np.errstate(over="ignore", invalid="ignore"):
        delta = logp - host(old).astype(np.float64)  # as fp32 holds old
        r = np.exp(delta)
        a = host(adv).astype(np.float64)
        free = np.where(a == 0, 0.0, r * a)
        cut = np.clip(r, 1 - CLIP[0], 1 + CLIP[1]) * a
    row = -np.minimum(free, cut)
    slope = np.where(free <= cut, -free, 0.0)
    rel = S + 12 * U
    dx = _grad(slope, 0.25, q, host(tok))
    dx_rel = (rel[:, None] + S[:, None] + U * (3 * zz + 14))
    # the token's own entry is 1 - q: both terms' errors beside what is left of them
    hot = np.arange(V) == host(tok)[:, None]
    dx_rel = np.where(hot, rel[:, None] + dx_rel * q / np.maximum(1 - q, 1e-12), dx_rel)
    with np.errstate(invalid="ignore"):
        row_tol = np.where(np.isfinite(row), np.abs(row) * rel, 0.0)
    got = M.policy_loss(x, tok, old, adv, clip=CLIP, weight=w, with_grad=True, grad_dtype=DT[dt])
    _check(got, row, row_tol, dx, dx_rel, dt)
    back = M.policy_loss_backward(x, got[3], tok, old, adv, clip=CLIP, weight=w, grad_dtype=DT[dt])
    assert torch.equal(back, got[4])
    up = a >= 0  # of these no loss is infinite
    some = torch.from_numpy(np.flatnonzero(up)).to(dev)
    part = M.policy_loss(x[some], tok[some], old[some], adv[some], clip=CLIP, weight=w[some])
    assert abs(float(part[0]) - 0.25 * row[up].sum()) <= 0.25 * (row_tol[up].sum() + 4 * U * np.abs(row[up]).sum())


@pytest.mark.parametrize("kl", [0.05, 1e-12])
def test_kl_term_far_from_the_reference(kl):
    dev = need_gpu()
    D = [d for d in DIFF if np.isfinite(d)] + [-600.0, -float("inf"), 0.49, 0.51, -0.51]
    T, V = len(D), 900
    x, tok, logp, q, zz, S = _rows(V, T, "f32", dev)
    ref = torch.from_numpy((logp + np.array(D)).astype(np.float32)).to(dev)
    zero = torch.zeros(T, device=dev)
    w = torch.full((T,), 0.25, device=dev)
    with np.errstate(over="ignore"):
        d = host(ref).astype(np.float64) - logp
        row, slope = kl * (np.expm1(d) - d), -kl * np.expm1(d)
    err = S + 4 * U
    with np.errstate(over="ignore", invalid="ignore"):
        row_tol = kl * (np.abs(np.expm1(d)) * err + 8 * U * np.where(np.abs(d) < 0.5, np.expm1(d) - d, np.exp(d) + 1))
        row_tol = np.where(np.isfinite(row), row_tol + 4 * U * np.abs(row), 0.0)
        rel = (np.exp(d) * err + 8 * U * np.where(np.abs(d) < 0.5, np.abs(np.expm1(d)), np.exp(d) + 1)) / np.abs(np.expm1(d))
    dx = _grad(slope, 0.25, q, host(tok))
    rel = np.nan_to_num(rel, nan=16 * U + err.max())
    dx_rel = rel[:, None] + S[:, None] + U * (3 * zz + 14)
    hot = np.arange(V) == host(tok)[:, None]
    dx_rel = np.where(hot, rel[:, None] + dx_rel * q / np.maximum(1 - q, 1e-12), dx_rel)
    got = M.policy_loss(x, tok, logp_old := ref.clone().fill_(-1.0), zero, ref_logp=ref, kl=kl, weight=w,
                        with_grad=True)
    _check(got, row, row_tol, dx, dx_rel, "f32")
    back = M.policy_loss_backward(x, got[3], tok, logp_old, zero, ref_logp=ref, kl=kl, weight=w)
    assert torch.equal(back, got[4])


def test_token_of_probability_zero():
    """A token that the mask excludes: its log-probability is -inf and its ratio 0; with a
    finite reference the KL term is infinite, the gradient finite."""
    dev = need_gpu()
    x, tok, *_ = _rows(300, 4, "f32", dev)
    tok[:] = 299
    adv = torch.tensor([1.0, 0.0, -1.0, 0.0], device=dev)
    old = torch.tensor([-3.0, -3.0, -3.0, -200.0], device=dev)
    loss, row, logp, stats, dx = M.policy_loss(x, tok, old, adv, clip=CLIP, with_grad=True)
    assert torch.isneginf(logp).all() and row[:2].tolist() == [0, 0] and abs(float(row[2]) - 0.8) < 1e-6 and row[3] == 0
    assert not dx.any()
    row, dx = (M.policy_loss(x, tok, old, adv, ref_logp=old, kl=0.1, with_grad=True)[i] for i in (1, 4))
    assert torch.isposinf(row).all() and torch.isfinite(dx).all() and (dx[:, 299] < 0).all() and (dx[:, 280] == 0).all()


def test_a_gradient_factor_of_zero_and_a_nan():
    """grad_loss 0 beside an infinite ratio gives zeros; NaN stays NaN."""
    dev = need_gpu()
    x, tok, logp, *_ = _rows(300, 3, "f32", dev)
    old = torch.tensor([-float("inf"), 0.0, float("nan")], device=dev)
    adv = torch.tensor([-1.0, float("nan"), 0.0], device=dev)
    got = M.policy_loss(x, tok, old, adv, with_grad=True, grad_loss=torch.zeros(1, device=dev))
    assert torch.isposinf(got[1][0]) and not got[4][0].any()
    got = M.policy_loss(x, tok, old, adv, with_grad=True)
    assert torch.isnan(got[1][1:]).all() and torch.isnan(got[4][1:]).all() and torch.isfinite(got[4][0]).all()


def test_large_advantages_and_kl_weights():
    """Products that fp32 does not hold before the row's weight: 1e38 times a ratio of
    e^39 at a weight of 1e-30, and a KL weight beyond fp32."""
    dev = need_gpu()
    x, tok, logp, q, zz, S = _rows(300, 4, "f32", dev)
    at = torch.from_numpy(logp.astype(np.float32)).to(dev)
    adv = torch.tensor([-1e38, 1e38, -1e25, 0.0], device=dev)
    old = at - 39
    w = torch.full((4,), 1e-30, device=dev)
    hot = np.arange(300) == host(tok)[:, None]

    def rel_of(rel):
        r = rel[:, None] + S[:, None] + U * (3 * zz + 14)
        return np.where(hot, rel[:, None] + r * q / np.maximum(1 - q, 1e-12), r)

    wide = float(np.float32(1e-30))
    got = M.policy_loss(x, tok, old, adv, clip=CLIP, weight=w, with_grad=True)
    a, r = host(adv).astype(np.float64), np.exp(logp - host(old).astype(np.float64))
    slope = np.where(a < 0, -r * a, 0.0)
    dx = _grad(slope, wide, q, host(tok))
    row = np.where(a < 0, -r * a, -(1 + CLIP[1]) * a)
    _check(got, row, np.abs(row) * (S + 12 * U), dx, rel_of(S + 12 * U), "f32")
    none = M.policy_loss(x, tok, old, adv, clip=CLIP, weight=w, with_grad=True, grad_loss=torch.zeros(1, device=dev))
    assert not none[4].any()
    ref, kl = at + 1, 1e39
    d = host(ref).astype(np.float64) - logp
    got = M.policy_loss(x, tok, at, adv * 0, ref_logp=ref, kl=kl, weight=w, with_grad=True)
    dx = _grad(-kl * np.expm1(d), wide, q, host(tok))
    rel = (np.exp(d) * (S + 4 * U) + 8 * U * (np.exp(d) + 1)) / np.expm1(d)
    _check(got, kl * (np.expm1(d) - d), np.zeros(4), dx, rel_of(rel), "f32")
    none = M.policy_loss(x, tok, at, adv * 0, ref_logp=ref, kl=kl, weight=w, with_grad=True,
                         grad_loss=torch.zeros(1, device=dev))
    assert not none[4].any()
