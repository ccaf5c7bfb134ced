"""Pins for the oracle's layer norm, balance loss and AdamW: hand examples,
torch.autograd in fp64 over the definitions, central differences."""
import numpy as np
import pytest
import torch

from oracle import adamw as OA, balance_loss as OL, norm as ON


def _t(a, grad=True):
    return torch.tensor(np.asarray(a, dtype=np.float64), requires_grad=grad)


# ---------------------------------------------------------------- layer norm

def test_norm_hand_example():
    y, mean, rstd = ON.forward([[1.0, 3.0]], [2.0, 10.0], [0.5, -1.0], eps=0.0)
    assert mean[0] == 2.0 and rstd[0] == 1.0
    assert np.allclose(y, [[-1 * 2 + 0.5, 1 * 10 - 1.0]])


def test_norm_constant_row():
    y, mean, rstd = ON.forward(np.full((1, 5), 7.0), np.ones(5), np.arange(5.0), eps=1e-2)
    assert np.allclose(y[0], np.arange(5.0)) and np.isclose(rstd[0], 10.0) and mean[0] == 7.0


@pytest.mark.parametrize("rows,d,res", [(1, 1, False), (4, 7, True), (9, 33, False), (0, 5, True)])
def test_norm_backward_autograd(rows, d, res):
    rng = np.random.default_rng(rows * 100 + d)
    s, w, b, dy = rng.normal(size=(rows, d)) + 3, rng.normal(size=d), rng.normal(size=d), rng.normal(size=(rows, d))
    ds = rng.normal(size=(rows, d)) if res else None
    y, mean, rstd = ON.forward(s, w, b)
    ts, tw, tb = _t(s), _t(w), _t(b)
    c = ts - ts.mean(1, keepdim=True)
    ty = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * tw + tb
    assert np.allclose(ty.detach().numpy(), y)
    total = (ty * _t(dy, False)).sum() + (0 if ds is None else (ts * _t(ds, False)).sum())
    gs, gw, gb = torch.autograd.grad(total, (ts, tw, tb))
    dx, dw, db = ON.backward(dy, s, w, mean, rstd, ds)
    for a, g in ((dx, gs), (dw, gw), (db, gb)):
        assert np.allclose(a, g.numpy(), atol=1e-9, rtol=1e-9)


def test_norm_backward_differences():
    rng = np.random.default_rng(3)
    s, w, b, dy = rng.normal(size=(3, 11)), rng.normal(size=11), rng.normal(size=11), rng.normal(size=(3, 11))
    _, mean, rstd = ON.forward(s, w, b)
    dx, dw, db = ON.backward(dy, s, w, mean, rstd)
    h = 1e-6
    loss = lambda s_, w_, b_: float((ON.forward(s_, w_, b_)[0] * dy).sum())  # noqa: E731
    for _ in range(5):
        u, uw, ub = rng.normal(size=s.shape), rng.normal(size=11), rng.normal(size=11)
        num = (loss(s + h * u, w + h * uw, b + h * ub) - loss(s - h * u, w - h * uw, b - h * ub)) / (2 * h)
        assert np.isclose(num, (dx * u).sum() + (dw * uw).sum() + (db * ub).sum(), rtol=1e-6)


# ---------------------------------------------------------------- balance loss

def test_balance_uniform_and_collapsed():
    """Equal affinities: P = 1/E, and sum_e f = E, so the loss is alpha whatever
    the counts.  All tokens and all probability on one expert (k = 1): alpha E."""
    T, E = 12, 4
    idx = np.zeros((T, 1), dtype=np.int32)
    loss, counts, prob, _ = OL.forward(np.zeros((T, E)), idx, 0.5)
    assert np.isclose(loss, 0.5) and counts.tolist() == [[12, 0, 0, 0]] and np.allclose(prob, 0.25)
    L = np.full((T, E), -1e4)
    L[:, 0] = 3.0
    assert np.isclose(OL.forward(L, idx, 0.5)[0], 0.5 * E)


def test_balance_counts_by_hand():
    idx = np.array([[0, 1], [2, 0], [1, 2], [0, -1], [3, 3]], dtype=np.int32)
    off, mask = [1, 3, 3, 5], [1, 1, 0, 1, 1]
    loss, counts, prob, dprob = OL.forward(np.zeros((5, 4)), idx, 3.0, off, mask)
    assert counts.tolist() == [[1, 0, 1, 0], [0, 0, 0, 0], [1, 0, 0, 2]]
    assert np.allclose(prob, [[0.25] * 4, [0] * 4, [0.25] * 4])
    assert np.allclose(dprob[0], [2, 0, 2, 0]) and not dprob[1].any()
    assert np.allclose(dprob[2], [0.5, 0, 0, 1.0])
    assert np.isclose(loss, 3.0 / 3 * (4 * 2 / 2 / 4 + 4 * 3 / 4 / 4))


@pytest.mark.parametrize("ragged", [False, True])
def test_balance_backward_autograd_and_differences(ragged):
    rng = np.random.default_rng(7)
    T, E, k = 14, 6, 2
    L = rng.normal(size=(T, E)) * 3
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    off = [1, 5, 5, 13] if ragged else None
    mask = (rng.random(T) > 0.3) if ragged else None
    loss, _, _, dprob = OL.forward(L, idx, 0.7, off, mask)
    extra = rng.normal(size=(T, E))
    dl = OL.backward(L, dprob, off, mask, 1.5, extra) - extra
    tl = _t(L)
    a = torch.sqrt(torch.logaddexp(tl, torch.zeros_like(tl)))
    p = a / a.sum(1, keepdim=True)
    total, bounds = 0.0, off or [0, T]
    for s in range(len(bounds) - 1):
        for t in range(bounds[s], bounds[s + 1]):
            if mask is None or mask[t]:
                total = total + (p[t] * _t(dprob[s], False)).sum()
    assert np.isclose(float(total.detach()), loss)  # the loss is linear in p
    g, = torch.autograd.grad(1.5 * total, tl)
    assert np.allclose(dl, g.numpy(), rtol=1e-9, atol=1e-12)
    h, u = 1e-6, rng.normal(size=(T, E))
    num = (OL.forward(L + h * u, idx, 0.7, off, mask)[0] - OL.forward(L - h * u, idx, 0.7, off, mask)[0]) / (2 * h)
    assert np.isclose(1.5 * num, (dl * u).sum(), rtol=1e-5)


def test_balance_backward_extremes():
    L = np.array([[-1e4, -1e4], [800.0, -800.0]])
    dl = OL.backward(L, np.array([[1.0, 0.0]]))
    assert np.isfinite(dl).all() and not dl[0].any()


# ---------------------------------------------------------------- AdamW

H = dict(lr=1e-2, b1=0.9, b2=0.99, eps=1e-8, wd=0.1)


def test_adamw_first_step_by_hand():
    """From zero states the bias correction cancels: the update is lr sign(g)."""
    w, m, v, r = OA.step([1.0, -2.0], [0.5, -4.0], [0, 0], [0, 0], t=1, **H)
    assert np.allclose(w, [1 * (1 - 1e-3) - 1e-2, -2 * (1 - 1e-3) + 1e-2], rtol=1e-6)
    assert np.allclose(m, [0.05, -0.4]) and np.allclose(v, [0.0025, 0.16]) and np.allclose(r, [0.05, 0.4])


@pytest.mark.parametrize("t", [1, 2, 1000])
def test_adamw_sequence_against_fp64(t):
    rng = np.random.default_rng(t)
    w, g, m = (rng.normal(size=500).astype(np.float32) for _ in range(3))
    v = (rng.random(500) * 2).astype(np.float32)
    got = OA.step(w, g, m, v, t=t, scale=0.25, **H)
    ref = OA.exact(w, g, m, v, t=t, scale=0.25, **H)
    for a, b in zip(got, ref):
        assert np.abs(a - b).max() <= 1e-6 * np.abs(b).max()


def test_adamw_codes():
    rng = np.random.default_rng(5)
    x = (rng.normal(size=300) * np.exp(rng.normal(size=300) * 4)).astype(np.float32)
    x[130], x[131], x[299] = np.inf, np.nan, 0.0
    codes, scales = OA.encode(x)
    back = OA.decode(codes, scales)
    assert scales.size == 3 and (np.log2(scales) % 1 == 0).all()
    for i in range(3):
        t = x[i * 128:(i + 1) * 128]
        amax = np.abs(t[np.isfinite(t)]).max()
        assert amax <= 448 * scales[i] and amax > 224 * scales[i]
    fin = np.isfinite(x)
    assert np.isnan(back[~fin]).all()
    step = np.repeat(scales, 128)[:300]
    # nearest code: within 2^-4 relative, or half the subnormal step 2^-9
    assert (np.abs(back - x)[fin] <= np.maximum(np.abs(x) * 2.0 ** -4, step * 2.0 ** -10)[fin]).all()
    codes, scales = OA.encode(np.zeros(5, dtype=np.float32))
    assert not codes.any() and scales.tolist() == [1.0]
    assert OA.tile_scale(np.float32(448)) == 1 and OA.tile_scale(np.float32(448.00003)) == 2
    assert OA.tile_scale(np.float32(1e-38)) == np.float32(2.0 ** -100)
