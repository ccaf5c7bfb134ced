"""GPU parity: the distillation and policy losses and their gradients against the
fp64 oracle.

Tolerances, from the operations' roundings (U = 2^-24, z = (x - max)/tau):
  e = 2^((x - max) c): a difference, a product and the rounded c give 3 U |z|
      relative, the exponential itself 2 U; where a thread's sum is brought to
      the row's maximum that comes once more.
  sum: at most 8 + 16 + 10 additions; a thread's maximum grows in at most 4 steps,
      each with an exponential and a product (3 U; its own |z| is part of the 6 Z
      below, as the steps add up to at most |z|); past what the registers hold one
      addition and one such step per piece, V / 4096 of them: A U relative with
      A = 34 + 12 + 4 V / 4096; the e's errors average to (6 Z + 4) U with
      Z = sum e |z| / sum.  Together S.
  ln of a sum: S absolute, and 4 U its own.
  teacher's probabilities: (3 |z| + 2 + 12 + 6 Zt + 4) U relative, as above with
      at most 12 additions.
  row loss (distill): sum p (relative error of p) |log p - log q| + S + St + 8 U
      + U sum p |zt|, times tau^2, and its own rounding.
  logp: S + 4 U + U |logp|; the ratio the same and 6 U relative, the KL term's
      slope expm1(d) times that and 8 U of itself.
  gradient: k q (3 |z| + 8) U + k q S + k p (p's) + 4 U k (q + p) and for policy
      the slope's error, then the stored type's half step.
A row that does not count is exactly 0.
"""
import math

import numpy as np
import pytest
import torch

import moe_expert_routing_sqrt_amd as M
from oracle import vocab_loss as OV

from gpu_util import host, need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": U, "bf16": 2.0 ** -8}
TYPES = [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")]

# widths: below a piece, at and around the shapes' limits of both types, and past
# what a row's threads hold (131072 bf16, 65536 fp32)
SIZES = [(1, 1), (3, 2), (2, 7), (5, 8), (4, 9), (7, 100), (9, 512), (5, 1023), (6, 1025), (3, 4096), (4, 4099),
         (5, 8200), (3, 16385), (300, 33), (3, 32768), (3, 32769), (2, 65536), (2, 70001), (2, 131072), (2, 140003)]
SIZES += [(4, 5001), (3, 6144), (3, 6149), (2, 12288), (2, 12297), (2, 24577), (2, 49159), (2, 98311)]  # more limits


def _at(t, shift):
    s = torch.empty(t.numel() + shift, dtype=t.dtype, device=t.device)
    s[shift:] = t.reshape(-1)
    return s[shift:].view(t.shape)


def _logits(g, T, V, dt, dev, scale=3.0):
    x = scale * torch.randn(T, V, generator=g, device=dev) + 5 * torch.randn(T, 1, generator=g, device=dev)
    if V > 20:
        x[:, V - V // 10:] = float("-inf")  # a padded vocabulary
    return _at(x.to(DT[dt]), (T + V) % 3)


def _row_stats(x, tau):
    """per row: z [V], q, S (the sum's relative error)"""
    V = x.shape[1]
    m = x.max(1, keepdims=True)
    z = (x - m) / tau
    e = np.exp(z)
    s = e.sum(1, keepdims=True)
    zz = np.where(e > 0, np.abs(z), 0.0)
    S = U * (46 + V / 1024 + 6 * (e * zz).sum(1, keepdims=True) / s + 4)
    return zz, e / s, S


def _close(got, ref, tol, what):
    got, ref, tol = np.asarray(host(got), dtype=np.float64), np.asarray(ref), np.asarray(tol)
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= tol + 1e-37)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.abs(got - ref).max()}, allowed {np.max(tol)}"


def _check_distill(x, idx, t, tau, w, grad, got, dx, dt):
    xh, ih, th, wh = host(x).astype(np.float64), host(idx), host(t).astype(np.float64), None if w is None else host(w)
    T, V = xh.shape
    ref = OV.distill(xh, ih, th, tau, wh, grad)
    wts = np.full(T, 1.0 / T) if wh is None else wh
    row_tol, stat_tol, dx_tol = np.zeros(T), np.zeros((T, 2)), np.zeros((T, V))
    zz, q, S = _row_stats(xh, tau)
    for r in range(T):
        ok, p, logp = OV.teacher_row(ih[r], th[r], V, tau)
        if wts[r] == 0 or len(ok) == 0:
            continue
        zt = np.where(p > 0, np.abs((th[r][ok] - th[r][ok].max()) / tau), 0)
        St = U * (12 + 6 * (p * zt).sum() + 4)
        rel = U * (3 * zt + 2) + St
        some = p > 0
        with np.errstate(divide="ignore"):
            gap = np.abs(logp - np.log(q[r][ih[r][ok]]))
        row_tol[r] = tau ** 2 * ((p * rel)[some] @ gap[some] + S[r, 0] + St + 8 * U + U * p @ zt)
        row_tol[r] += U * abs(ref["row_loss"][r])
        stat_tol[r, 1] = S[r, 0] * ref["stats"][r, 1]
        k = abs(grad * wts[r] * tau)
        d = q[r] * (U * (3 * zz[r] + 12) + S[r])
        np.add.at(d, ih[r][ok], p * (rel + 8 * U))
        dx_tol[r] = k * d
    if got is not None:
        loss, row, stats = got
        _close(row, ref["row_loss"], row_tol, "row_loss")
        _close(stats, ref["stats"], stat_tol, "stats")
        live = wts != 0
        _close(loss, [ref["loss"]], [(np.abs(wts) * row_tol)[live].sum() + 2 * U * abs(ref["loss"])
                                     + U * (np.abs(wts * ref["row_loss"]))[live].sum()], "loss")
    if dx is not None:
        _close(dx, ref["dlogits"], dx_tol + HALF[dt] * (np.abs(ref["dlogits"]) + dx_tol), "dlogits")


def _teacher(g, x, K, dev, ragged=True):
    T, V = x.shape
    idx = torch.randint(0, V, (T, K), generator=g, device=dev)
    best = x.float().argmax(1)
    idx[:, 0] = best                                        # the likeliest token among them
    if K > 3:
        idx[:, 3] = idx[:, 0]                               # and once more
    t = torch.gather(x.float(), 1, idx).clamp(min=-20) + torch.randn(T, K, generator=g, device=dev)
    idx = idx.to(torch.int32)
    if ragged and K > 1:
        keep = torch.randint(0, K + 1, (T, 1), generator=g, device=dev)
        idx = torch.where(torch.arange(K, device=dev) < keep, idx, torch.where(keep % 2 == 0, -1, V + 3)).to(torch.int32)
        t[:, K - 1] = float("-inf")
    # a teacher's token that the student's vocabulary masks has no finite loss
    masked = torch.isinf(torch.gather(x.float(), 1, idx.clamp(0, V - 1).long()))
    return torch.where(masked, -1, idx).contiguous(), t


@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("xt,dt", TYPES)
def test_distill(T, V, xt, dt):
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(T * 7 + V)
    K = [1, 5, 64, 65, 200, 256][(T + V) % 6]
    tau = [1.0, 2.0, 0.7][V % 3]
    print(f"distill {T}x{V} K={K} tau={tau} {xt}->{dt}", flush=True)
    x = _logits(g, T, V, xt, dev)
    idx, t = _teacher(g, x, K, dev)
    if V % 2:
        t = t.to(torch.bfloat16)
    w = None if T % 2 else torch.rand(T, generator=g, device=dev) * (torch.rand(T, generator=g, device=dev) > 0.3)
    gl = torch.full((1,), 3.0, device=dev)
    loss, row, stats, none = M.distill_loss(x, idx, t, tau, w)
    assert none is None
    _check_distill(x, idx, t, tau, w, 1.0, (loss, row, stats), None, dt)
    one = M.distill_loss(x, idx, t, tau, w, with_grad=True, grad_loss=gl, grad_dtype=DT[dt])
    assert all(torch.equal(a, b) for a, b in zip((loss, row, stats), one))
    _check_distill(x, idx, t, tau, w, 3.0, None, one[3], dt)
    two = M.distill_loss_backward(x, stats, idx, t, tau, w, grad_loss=gl, grad_dtype=DT[dt])
    assert torch.equal(one[3], two)  # both evaluate the same expression
    if xt == dt:
        y = x.clone()
        assert M.distill_loss(y, idx, t, tau, w, dlogits=y, grad_loss=gl)[3] is y
        assert torch.equal(y, two)


def _check_policy(x, tok, old, adv, ref_logp, clip, kl, tau, w, grad, got, dx, dt):
    xh, th, wh = host(x).astype(np.float64), host(tok), None if w is None else host(w)
    T, V = xh.shape
    args = (th, host(old), host(adv), None if ref_logp is None else host(ref_logp), clip, kl, tau, wh)
    ref = OV.policy(xh, *args, grad=grad)
    wts = np.full(T, 1.0 / T) if wh is None else wh
    row_tol, lp_tol, stat_tol, dx_tol = np.zeros(T), np.zeros(T), np.zeros((T, 2)), np.zeros((T, V))
    zz, q, S = _row_stats(xh, tau)
    for r in range(T):
        if wts[r] == 0 or not 0 <= th[r] < V:
            continue
        lp, a, o = ref["logp"][r], float(host(adv)[r]), float(host(old)[r])
        err = S[r, 0] + 4 * U
        lp_tol[r] = err + U * abs(lp)
        ratio = math.exp(lp - o)
        rel = err + U * (6 + abs(lp - o))
        row_tol[r] = ratio * abs(a) * (rel + 2 * U)
        slope_tol = row_tol[r]
        slope = -ratio * a if ratio * a <= min(max(ratio, 1 - clip[0]), 1 + clip[1]) * a else 0.0
        if kl:
            d = float(host(ref_logp)[r]) - lp
            e1, k3 = math.expm1(d), math.expm1(d) - d
            row_tol[r] += kl * (abs(e1) * (err + U * abs(d)) + 8 * U * (k3 if abs(d) < 0.5 else math.exp(d) + abs(d) + 1))
            slope_tol += kl * (math.exp(d) * (err + U * abs(d)) + 8 * U * (abs(e1) if abs(d) < 0.5 else math.exp(d) + 1))
            slope -= kl * e1
        row_tol[r] += 2 * U * abs(ref["row_loss"][r])
        stat_tol[r, 1] = S[r, 0] * ref["stats"][r, 1]
        k = abs(grad * wts[r] / tau)
        hot = np.arange(V) == th[r]
        dx_tol[r] = k * abs(slope) * (q[r] * (U * (3 * zz[r] + 14) + S[r]) + 8 * U * hot) + k * slope_tol * (q[r] + hot)
    if got is not None:
        loss, row, logp, stats = got
        _close(row, ref["row_loss"], row_tol, "row_loss")
        _close(logp, ref["logp"], lp_tol, "logp")
        _close(stats, ref["stats"], stat_tol, "stats")
        live = wts != 0
        _close(loss, [ref["loss"]], [(np.abs(wts) * row_tol)[live].sum() + 2 * U * abs(ref["loss"])
                                     + U * (np.abs(wts * ref["row_loss"]))[live].sum()], "loss")
    if dx is not None:
        _close(dx, ref["dlogits"], dx_tol + HALF[dt] * (np.abs(ref["dlogits"]) + dx_tol), "dlogits")


def _rollout(g, x, tau, dev, clip=(0.2, 0.28)):
    """tokens, old and reference log-probabilities (ratios inside, outside and off the
    clip's borders), advantages"""
    T, V = x.shape
    z = x.double() / tau
    gum = -torch.log(-torch.log(torch.rand(T, V, generator=g, device=dev).double().clamp(1e-12, 1 - 1e-12)))
    tok = (z + gum).argmax(1)
    logp = torch.log_softmax(z, 1).gather(1, tok[:, None])[:, 0]
    move = 0.4 * torch.randn(T, generator=g, device=dev).double()
    for b in (math.log(1 - clip[0]), math.log(1 + clip[1])):
        move = torch.where((move - b).abs() < 1e-3, move + 4e-3, move)
    ref = logp + torch.randn(T, generator=g, device=dev) * torch.tensor([1.0, 1e-3, 0.0], device=dev)[torch.arange(T, device=dev) % 3]
    return tok.to(torch.int32), (logp - move).float(), torch.randn(T, generator=g, device=dev), ref.float(), logp


@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("xt,dt", TYPES)
def test_policy(T, V, xt, dt):
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(T * 5 + V)
    tau, kl = [1.0, 2.0, 0.7][V % 3], [0.0, 0.3][T % 2]
    print(f"policy {T}x{V} tau={tau} kl={kl} {xt}->{dt}", flush=True)
    x = _logits(g, T, V, xt, dev)
    tok, old, adv, ref, logp = _rollout(g, x, tau, dev)
    w = None
    if T > 2:
        tok[1], tok[2] = -1, V
        w = torch.rand(T, generator=g, device=dev) * (torch.rand(T, generator=g, device=dev) > 0.3)
    gl = torch.full((1,), -2.0, device=dev)
    kw = dict(ref_logp=ref if kl else None, clip=(0.2, 0.28), kl=kl, temperature=tau, weight=w)
    *got, none = M.policy_loss(x, tok, old, adv, **kw)
    assert none is None
    args = (x, tok, old, adv, ref, (0.2, 0.28), kl, tau, w)
    _check_policy(*args, 1.0, got, None, dt)
    one = M.policy_loss(x, tok, old, adv, **kw, with_grad=True, grad_loss=gl, grad_dtype=DT[dt])
    assert all(torch.equal(a, b) for a, b in zip(got, one))
    _check_policy(*args, -2.0, None, one[4], dt)
    two = M.policy_loss_backward(x, got[3], tok, old, adv, **kw, grad_loss=gl, grad_dtype=DT[dt])
    assert torch.equal(one[4], two)
    if xt == dt:
        y = x.clone()
        assert M.policy_loss(y, tok, old, adv, **kw, dlogits=y, grad_loss=gl)[4] is y
        assert torch.equal(y, two)
    if w is None:
        lp, st = M.token_logp(x, tok, tau)
        assert torch.equal(lp, got[2]) and torch.equal(st, got[3])


def test_gradients_by_differences():
    """Directional central differences of the losses, along a random direction."""
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(11)
    T, V, K, h = 40, 500, 12, 2.0 ** -7
    x = torch.randn(T, V, generator=g, device=dev)
    u = torch.randn(T, V, generator=g, device=dev)
    idx, t = _teacher(g, x, K, dev, ragged=False)
    up, down = (M.distill_loss(x + s * h * u, idx, t, 1.5)[1].double() for s in (1, -1))
    dx = M.distill_loss(x, idx, t, 1.5, weight=torch.ones(T, device=dev), with_grad=True)[3].double()
    # third derivatives of a log-sum-exp are at most 1 in |u|_inf^3 / 6 h^2; fp32 losses carry 1e-5 / h
    bound = h * h / 6 * u.abs().amax(1).double() ** 3 * 8 + 1e-5 / h
    assert ((up - down) / (2 * h) - (dx * u).sum(1)).abs().le(bound).all()
    tok, old, _, _, logp = _rollout(g, x, 1.0, dev)
    adv = torch.ones(T, device=dev)
    kw = dict(clip=(0.9, 50.0), kl=0.0)  # no clipping near the ratios
    up, down = (M.policy_loss(x + s * h * u, tok, old, adv, **kw)[1].double() for s in (1, -1))
    dx = M.policy_loss(x, tok, old, adv, **kw, weight=adv, with_grad=True)[4].double()
    bound = (h * h * u.abs().amax(1).double() ** 3 * 8 + 1e-5 / h) * torch.exp(logp - old.double()) * 2
    assert ((up - down) / (2 * h) - (dx * u).sum(1)).abs().le(bound).all()


def test_rows_that_do_not_count_may_hold_anything():
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(2)
    for V in (100, 9000, 40000):
        T = 6
        x = torch.randn(T, V, generator=g, device=dev)
        idx, t = _teacher(g, x, 4, dev, ragged=False)
        clean = M.distill_loss(x, idx, t, weight=torch.tensor([0, 1, 0, 1, 1, 1.0], device=dev), with_grad=True)
        y = x.clone()
        y[0], y[2, 5] = float("nan"), float("inf")
        w = torch.tensor([0, 1, 0, 1, 1, 1.0], device=dev)
        got = M.distill_loss(y, idx, t, weight=w, with_grad=True)
        assert all(torch.equal(a, b) for a, b in zip(clean, got))
        assert not got[3][0].any() and not got[2][0].any() and got[1][0] == 0
        # no teacher entry: out of range, or all of them -inf
        i2, t2 = idx.clone(), t.clone()
        i2[0], t2[2] = -1, float("-inf")
        got = M.distill_loss(y, i2, t2, with_grad=True)
        assert torch.isfinite(got[0]) and torch.isfinite(got[3]).all()
        assert not got[3][0].any() and not got[3][2].any() and got[3][1].any()
        back = M.distill_loss_backward(y, got[2], i2, t2)
        assert torch.equal(back, got[3])
        tok = torch.tensor([-1, 3, V, 3, 3, 3], dtype=torch.int32, device=dev)
        o, a = torch.full((T,), -4.0, device=dev), torch.ones(T, device=dev)
        o[0], a[2] = float("nan"), float("nan")
        got = M.policy_loss(y, tok, o, a, ref_logp=o, kl=0.1, with_grad=True)
        assert torch.isfinite(got[0]) and torch.isfinite(got[4]).all() and got[1][0] == 0 and got[2][2] == 0
        assert not got[4][0].any() and not got[4][2].any() and got[4][1].any()
        assert torch.equal(M.policy_loss_backward(y, got[3], tok, o, a, ref_logp=o, kl=0.1), got[4])
        lp, _ = M.token_logp(y, tok)
        assert lp[0] == 0 and lp[2] == 0 and lp[1] == got[2][1]


def test_nan_and_infinity_stay_in_their_row():
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(3)
    for V in (64, 5000, 33000, 150000):
        x = torch.randn(5, V, generator=g, device=dev)
        x[1, V // 2], x[2, 0], x[3] = float("nan"), float("inf"), float("-inf")
        idx = torch.tensor([[1, 2]], dtype=torch.int32, device=dev).repeat(5, 1)
        t = torch.zeros(5, 2, device=dev)
        loss, row, _, dx = M.distill_loss(x, idx, t, with_grad=True)
        assert torch.isnan(loss).all() and torch.isnan(row[1:4]).all() and torch.isnan(dx[1:4]).all()
        assert torch.isfinite(row[[0, 4]]).all() and torch.isfinite(dx[[0, 4]]).all()
        tok = torch.ones(5, dtype=torch.int32, device=dev)
        z = torch.zeros(5, device=dev)
        loss, row, _, _, dx = M.policy_loss(x, tok, z - 3, z + 1, with_grad=True)
        assert torch.isnan(row[1:4]).all() and torch.isfinite(dx[[0, 4]]).all() and torch.isnan(dx[1:4]).all()
        # a NaN of the teacher
        t[4, 0] = float("nan")
        _, row, _, dx = M.distill_loss(x, idx, t, with_grad=True)
        assert torch.isnan(row[4]) and torch.isfinite(row[0])
        # the teacher wants what the student's mask excludes: an infinite loss, a finite gradient
        x[0, 2] = float("-inf")
        _, row, _, dx = M.distill_loss(x, idx, t, with_grad=True)
        assert row[0] == float("inf") and torch.isfinite(dx[0]).all() and dx[0, 2] < 0


def test_extreme_logits():
    """Rows at the types' ends: a constant row of the lowest value, and differences that
    overflow."""
    dev = need_gpu()
    for dt in (torch.float32, torch.bfloat16):
        low = torch.finfo(dt).min
        x = torch.zeros(3, 300, device=dev, dtype=dt)
        x[0] = low
        x[1], x[1, 7] = low, torch.finfo(dt).max
        x[2, 1:] = low
        tok = torch.tensor([5, 7, 0], dtype=torch.int32, device=dev)
        lp, st = M.token_logp(x, tok)
        assert abs(float(lp[0]) + math.log(300)) < 1e-6 and lp[1] == 0 and lp[2] == 0
        assert st[0, 1] == 300 and st[1, 1] == 1 and st[2, 1] == 1


@pytest.mark.parametrize("K", [1, 2, 63, 64, 130, 256])
def test_repeated_indices(K):
    """All entries the same token, in pairs, or neighbours in one thread's pieces."""
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(K)
    for V in (300, 40000):
        x = torch.randn(4, V, generator=g, device=dev)
        idx = torch.full((4, K), 17, dtype=torch.int32, device=dev)
        idx[1] = torch.arange(K, device=dev) // 2
        idx[2] = torch.arange(K, device=dev)
        idx[3] = V - 1 - torch.arange(K, device=dev) % 5
        t = torch.randn(4, K, generator=g, device=dev)
        got = M.distill_loss(x, idx, t, with_grad=True)
        _check_distill(x, idx, t, 1.0, None, 1.0, got[:3], got[3], "f32")
        for _ in range(5):
            assert all(torch.equal(a, b) for a, b in zip(got, M.distill_loss(x, idx, t, with_grad=True)))


@pytest.mark.parametrize("gap", [1e-1, 1e-3, 1e-5])
def test_small_losses(gap):
    """Student and teacher nearly the same: the loss is of the order gap^2, its error
    stays that of the logarithms."""
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(6)
    x = torch.randn(8, 32, generator=g, device=dev)
    idx = torch.arange(32, device=dev, dtype=torch.int32).repeat(8, 1)
    t = x + gap * torch.randn(8, 32, generator=g, device=dev)
    got = M.distill_loss(x, idx, t, with_grad=True)
    _check_distill(x, idx, t, 1.0, None, 1.0, got[:3], got[3], "f32")
    lp, _ = M.token_logp(x, idx[:, 0].contiguous())
    ref = (lp.double() + gap).float()
    tok, z = idx[:, 3].contiguous(), torch.zeros(8, device=dev)
    got = M.policy_loss(x, tok, lp, z, ref_logp=M.token_logp(x, tok)[0] + gap, kl=1.0, with_grad=True)
    _check_policy(x, tok, lp, z, M.token_logp(x, tok)[0] + gap, (0.2, 0.2), 1.0, 1.0, None, 1.0, got[:4], got[4], "f32")
    assert ref.shape == lp.shape


def test_many_rows_and_walks():
    """More rows than work-groups at once, some that do not count, of every shape."""
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(9)
    for T, V in ((20000, 40), (9000, 1500), (3000, 5000), (2500, 17000), (1100, 33000), (600, 70000)):
        x = torch.randn(T, V, generator=g, device=dev, dtype=torch.float32).to(torch.bfloat16)
        w = (torch.rand(T, generator=g, device=dev) > 0.3).float()
        tok = torch.randint(-V // 9, V, (T,), generator=g, device=dev, dtype=torch.int32)
        old, adv = torch.full((T,), -math.log(V), device=dev), torch.randn(T, generator=g, device=dev)
        print(f"rows {T}x{V}", flush=True)
        got = M.policy_loss(x, tok, old, adv, weight=w, clip=(0.5, 1.0), with_grad=True)
        rows = torch.cat([torch.arange(5), torch.randint(0, T, (20,)), torch.tensor([T - 1])]).to(dev)
        part = tuple(t[rows].contiguous() for t in (x, tok, old, adv))
        _check_policy(*part, None, (0.5, 1.0), 0.0, 1.0, w[rows].contiguous(), 1.0, None, got[4][rows], "bf16")
        sub = M.policy_loss(*part, weight=w[rows].contiguous(), clip=(0.5, 1.0), with_grad=True)
        for a, b in zip(sub[1:], got[1:]):
            assert torch.equal(a, b[rows])
        total = (w.double() * got[1].double()).sum()
        assert abs(float(got[0]) - float(total)) <= 2 * U * abs(float(total)) + 1e-12 * float((w * got[1].abs()).sum())


def test_past_32_bit_offsets():
    dev = need_gpu()
    T, V = 70000, 65536  # 4.6 G logits
    x = torch.zeros(T, V, dtype=torch.bfloat16, device=dev)
    x[T - 1, V - 1], x[66000, 3] = 5.0, 2.0
    tok = torch.full((T,), 3, dtype=torch.int32, device=dev)
    tok[T - 1] = V - 1
    w = torch.zeros(T, device=dev)
    w[T - 1] = w[66000] = 1.0
    z = torch.zeros(T, device=dev)
    _, row, logp, stats, dx = M.policy_loss(x, tok, z - math.log(V), z + 1, weight=w, clip=(1.0, 1e9), dlogits=x)
    want = torch.tensor([5.0 - math.log(V - 1 + math.exp(5.0)), 2.0 - math.log(V - 1 + math.exp(2.0))])
    assert (logp[[T - 1, 66000]].cpu() - want).abs().max() < 1e-5
    assert dx[T - 1, V - 1] < 0 and dx[66000, 3] < 0 and int((dx[:, 3] != 0).sum()) == 2


def test_equal_bits_on_every_call_streams_and_graphs():
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(5)
    T, V, K = 700, 20000, 40
    x = torch.randn(T, V, generator=g, device=dev).to(torch.bfloat16)
    idx, t = _teacher(g, x, K, dev)
    first = M.distill_loss(x, idx, t, with_grad=True)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(M.distill_loss(x, idx, t, with_grad=True), first))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for i in range(6):
        with torch.cuda.stream(s1 if i % 2 else s2):
            outs.append(M.distill_loss(x, idx, t, with_grad=True))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, first))
    tok, old, adv, ref, _ = _rollout(g, x[:, :-5].contiguous(), 1.0, dev)
    dx, loss = torch.empty_like(x), torch.empty(1, device=dev)
    row, logp, stats = (torch.empty(n, device=dev) for n in (T, T, 2 * T))
    d2 = torch.empty_like(x)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        M.policy_loss(x, tok, old, adv, ref, kl=0.1, loss=loss, row_loss=row, logp=logp, stats=stats, dlogits=dx)
        M.policy_loss_backward(x, stats, tok, old, adv, ref, kl=0.1, dlogits=d2)
    for _ in range(4):
        x.copy_(torch.randn(T, V, generator=g, device=dev))
        adv.copy_(torch.randn(T, generator=g, device=dev))
        gr.replay()
        torch.cuda.synchronize()
        e = M.policy_loss(x, tok, old, adv, ref, kl=0.1, with_grad=True)
        assert torch.equal(e[0], loss) and torch.equal(e[1], row) and torch.equal(e[2], logp)
        assert torch.equal(e[4], dx) and torch.equal(dx, d2)


def test_no_rows():
    dev = need_gpu()
    x = torch.zeros(0, 50, device=dev)
    i, f = torch.zeros(0, 3, dtype=torch.int32, device=dev), torch.zeros(0, 3, device=dev)
    loss, row, stats, dx = M.distill_loss(x, i, f, with_grad=True, loss=torch.full((1,), 9.0, device=dev))
    assert loss == 0 and row.shape == (0,) and dx.shape == (0, 50)
    loss, _, _, _, _ = M.policy_loss(x, i[:, 0].contiguous(), f[:, 0].contiguous(), f[:, 0].contiguous(),
                                     loss=torch.full((1,), 9.0, device=dev))
    assert loss == 0


def test_refusals():
    dev = need_gpu()
    x, i = torch.zeros(4, 8, device=dev), torch.zeros(4, dtype=torch.int32, device=dev)
    f = torch.zeros(4, device=dev)
    with pytest.raises(TypeError, match="idx must be int32"):
        M.distill_loss(x, i.long().view(4, 1), f.view(4, 1))
    with pytest.raises(ValueError, match="teacher: needs"):
        M.distill_loss(x, i.view(4, 1), f[:3].view(3, 1))
    with pytest.raises(TypeError, match="grad_dtype"):
        M.distill_loss(x, i.view(4, 1), f.view(4, 1), dlogits=x, grad_dtype=torch.bfloat16)
    with pytest.raises(M.MoeError):
        M.distill_loss(x, i.view(4, 1), f.view(4, 1), temperature=0.0)
    with pytest.raises(M.MoeError):
        M.distill_loss_backward(x, torch.zeros(4, 2, device=dev), i.view(4, 1), f.view(4, 1), dlogits=x)
    with pytest.raises(M.MoeError):
        M.policy_loss(x, i, f, f, kl=0.1)
    with pytest.raises(M.MoeError):
        M.policy_loss(x, i, f, f, clip=(-0.1, 0.2))
    with pytest.raises(TypeError, match="weight must be float32"):
        M.policy_loss(x, i, f, f, weight=f.bfloat16())
    with pytest.raises(TypeError):
        M.token_logp(x.half(), i)
    with pytest.raises(ValueError, match="contiguous"):
        M.token_logp(torch.zeros(8, 4, device=dev).t(), i)
