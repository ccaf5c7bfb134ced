"""Pins of the embedding and vocabulary-loss oracles: hand-computed rows, closed
forms, a pure-Python brute force, torch.autograd in fp64, central differences."""
import math

import numpy as np
import pytest
import torch

from oracle import embedding as OE, vocab_loss as OV


def test_embedding_by_hand():
    table = np.array([[1.0, 2.0], [3.0, -4.0], [0.5, 0.0]])
    ids = [2, -1, 0, 3, 2]
    assert np.array_equal(OE.forward(ids, table, 2.0), [[1, 0], [0, 0], [2, 4], [0, 0], [1, 0]])
    dy = np.array([[1.0, 1.0], [9, 9], [2, -1], [9, 9], [3, 0.5]])
    d, mags, n = OE.backward(dy, ids, 3, 2.0)
    assert np.array_equal(d, [[4, -2], [0, 0], [8, 3]]) and np.array_equal(mags, [[4, 2], [0, 0], [8, 3]])
    assert np.array_equal(n, [1, 0, 2])


def test_embedding_is_a_one_hot_product():
    g = np.random.default_rng(0)
    V, d, T = 13, 5, 40
    ids, table, dy = g.integers(-2, V + 2, T), g.standard_normal((V, d)), g.standard_normal((T, d))
    hot = (ids[:, None] == np.arange(V)).astype(float)
    assert np.allclose(OE.forward(ids, table, 0.3), 0.3 * hot @ table, rtol=1e-14, atol=1e-14)
    assert np.allclose(OE.backward(dy, ids, V, 0.3)[0], 0.3 * hot.T @ dy, rtol=1e-13, atol=1e-14)
    w = torch.tensor(table, requires_grad=True)
    ok = (ids >= 0) & (ids < V)
    (w[torch.tensor(ids[ok])] * 0.3 * torch.tensor(dy[ok])).sum().backward()
    assert np.allclose(w.grad.numpy(), OE.backward(dy, ids, V, 0.3)[0], rtol=1e-13, atol=1e-14)


def test_distill_two_logits_closed_form():
    # teacher all on entry 0: the loss is tau^2 log(1 + exp((x1 - x0)/tau))
    for tau in (1.0, 2.0, 0.5):
        r = OV.distill([[0.3, 1.1]], np.array([[0]]), [[5.0]], tau)
        gap = 0.8 / tau
        assert math.isclose(r["loss"], tau ** 2 * math.log1p(math.exp(gap)), rel_tol=1e-14)
        q1 = 1 / (1 + math.exp(-gap))
        assert np.allclose(r["dlogits"], [[-tau * q1, tau * q1]], rtol=1e-14)


def test_distill_zero_where_student_is_teacher():
    x = np.random.default_rng(1).standard_normal((3, 7))
    r = OV.distill(x, np.tile(np.arange(7), (3, 1)), x + 2.5, 1.7)
    assert np.abs(r["row_loss"]).max() < 1e-15 and np.abs(r["dlogits"]).max() < 1e-15


def test_policy_two_logits_closed_form():
    x = [[0.0, 0.0]]
    r = OV.policy(x, [1], [math.log(0.5)], [3.0])          # r = 1: l = -A
    assert math.isclose(r["loss"], -3.0) and np.allclose(r["dlogits"], [[1.5, -1.5]])
    up = OV.policy(x, [1], [math.log(0.25)], [3.0])        # r = 2, clipped above: no gradient
    assert math.isclose(up["loss"], -3.6) and not up["dlogits"].any()
    down = OV.policy(x, [1], [math.log(0.25)], [-3.0])     # r = 2, A < 0: not clipped
    assert math.isclose(down["loss"], 6.0) and np.allclose(down["dlogits"], [[-3.0, 3.0]])
    low = OV.policy(x, [1], [0.0], [-3.0])                 # r = 0.5, A < 0: clipped below
    assert math.isclose(low["loss"], 2.4) and not low["dlogits"].any()
    k = OV.policy(x, [1], [math.log(0.5)], [0.0], [math.log(0.25)], kl=2.0)  # exp(d) = 1/2
    assert math.isclose(k["loss"], 2 * (0.5 + math.log(2) - 1), rel_tol=1e-14)
    assert np.allclose(k["dlogits"], np.array([[-1, 1]]) * 2 * (1 - 0.5) * 0.5)


def _case(seed, T=6, V=11, K=5):
    g = np.random.default_rng(seed)
    x = 2 * g.standard_normal((T, V))
    idx = g.integers(-1, V + 1, (T, K))
    idx[1] = -1
    t = 2 * g.standard_normal((T, K))
    t[2, 0] = -np.inf
    w = g.random(T)
    w[3] = 0
    return g, x, idx, t, w


def test_distill_brute_force():
    _, x, idx, t, w = _case(2)
    r = OV.distill(x, idx, t, 1.3, w, 0.7)
    for i in range(len(x)):
        es = [math.exp(v / 1.3) for v in x[i]]
        ent = [(j, math.exp(v / 1.3)) for j, v in zip(idx[i], t[i]) if 0 <= j < x.shape[1] and v > -math.inf]
        if not ent or w[i] == 0:
            assert r["row_loss"][i] == 0 and not r["dlogits"][i].any() and not r["stats"][i].any()
            continue
        tot = sum(e for _, e in ent)
        l = sum(e / tot * (math.log(e / tot) - math.log(es[j] / sum(es))) for j, e in ent) * 1.69
        assert math.isclose(r["row_loss"][i], l, rel_tol=1e-12, abs_tol=1e-13)
        for v in range(x.shape[1]):
            p = sum(e for j, e in ent if j == v) / tot
            assert math.isclose(r["dlogits"][i, v], 0.7 * w[i] * 1.3 * (es[v] / sum(es) - p), rel_tol=1e-11,
                                abs_tol=1e-15)


def _differences(f, x, h=1e-6):
    d = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        d[i] = (f(up) - f(down)) / (2 * h)
    return d


def test_distill_gradient_by_differences_and_autograd():
    _, x, idx, t, w = _case(3)
    r = OV.distill(x, idx, t, 0.8, w)
    assert np.abs(_differences(lambda y: OV.distill(y, idx, t, 0.8, w)["loss"], x) - r["dlogits"]).max() < 1e-8
    X = torch.tensor(x, requires_grad=True)
    total = 0.0
    for i in range(len(x)):
        ok, p, logp = OV.teacher_row(idx[i], t[i], x.shape[1], 0.8)
        z = torch.log_softmax(X[i] / 0.8, 0)[torch.tensor(idx[i][ok])]
        total = total + w[i] * 0.64 * (torch.tensor(p) * (torch.tensor(logp) - z)).sum()
    total.backward()
    assert math.isclose(float(total.detach()), r["loss"], rel_tol=1e-12)
    assert np.allclose(X.grad.numpy(), r["dlogits"], rtol=1e-11, atol=1e-14)


@pytest.mark.parametrize("kl", [0.0, 0.3])
def test_policy_gradient_by_differences_and_autograd(kl):
    g, x, _, _, w = _case(4)
    T, V = x.shape
    tok = g.integers(0, V, T)
    tok[4] = V
    logp = np.array([OV.softmax_row(x[i], 1.5)[1][tok[i] % V] for i in range(T)])
    old, adv, ref = logp + 0.4 * g.standard_normal(T), g.standard_normal(T), logp + g.standard_normal(T)
    args = (tok, old, adv, ref, (0.2, 0.3), kl, 1.5, w)
    r = OV.policy(x, *args)
    assert np.abs(_differences(lambda y: OV.policy(y, *args)["loss"], x) - r["dlogits"]).max() < 1e-7
    X = torch.tensor(x, requires_grad=True)
    total = 0.0
    for i in range(T):
        if tok[i] >= V:
            assert not r["dlogits"][i].any() and r["logp"][i] == 0
            continue
        lp = torch.log_softmax(X[i] / 1.5, 0)[tok[i]]
        ratio = torch.exp(lp - old[i])
        l = -torch.minimum(ratio * adv[i], torch.clamp(ratio, 0.8, 1.3) * adv[i])
        l = l + kl * (torch.exp(ref[i] - lp) - (ref[i] - lp) - 1)
        total = total + w[i] * l
    total.backward()
    assert math.isclose(float(total.detach()), r["loss"], rel_tol=1e-12)
    assert np.allclose(X.grad.numpy(), r["dlogits"], rtol=1e-11, atol=1e-14)
