"""The token calls refuse outputs that share memory with each other or with what other
rows still read, wherever the shared part lies (no GPU: refused before any launch)."""
import ctypes

import pytest

from moe_expert_routing_sqrt_amd import _lib

L = _lib.load()
INV = _lib.MOE_ERR_INVALID_ARG
T, V, K, D = 64, 1000, 8, 32
# one region each, 1 MB apart: never dereferenced
X, I, TE, W, G, LO, RO, ST, DX, LP, O, A, R = (0x10000000 + (i << 20) for i in range(13))


def _distill(x=X, xt=0, idx=I, t=TE, w=W, g=G, loss=LO, row=RO, stats=ST, dx=DX, dt=0):
    return L.moe_distill_loss(T, V, K, x, xt, idx, t, 0, 1.0, w, g, loss, row, stats, dx, dt, None)


def _distill_bwd(x=X, xt=0, idx=I, t=TE, w=W, g=G, stats=ST, dx=DX, dt=0):
    return L.moe_distill_loss_backward(T, V, K, x, xt, stats, idx, t, 0, 1.0, w, g, dx, dt, None)


H = _lib.MoePolicyParams(1.0, 0.2, 0.2, 0.1)


def _policy(x=X, xt=0, tok=I, old=O, adv=A, ref=R, w=W, g=G, loss=LO, row=RO, logp=LP, stats=ST, dx=DX, dt=0):
    return L.moe_policy_loss(T, V, x, xt, tok, old, adv, ref, ctypes.byref(H), w, g, loss, row, logp, stats, dx, dt, None)


def _policy_bwd(x=X, xt=0, tok=I, old=O, adv=A, ref=R, w=W, g=G, stats=ST, dx=DX, dt=0):
    return L.moe_policy_loss_backward(T, V, x, xt, stats, tok, old, adv, ref, ctypes.byref(H), w, g, dx, dt, None)


def _logp(x=X, tok=I, logp=LP, stats=ST):
    return L.moe_token_logp(T, V, x, 0, tok, 1.0, logp, stats, None)


SHARED = [dict(row=LO), dict(stats=RO), dict(loss=ST), dict(stats=RO + 4 * T - 4), dict(row=ST + 8 * T - 4),
          dict(loss=RO + 4 * T - 4), dict(row=X + 40), dict(stats=DX + 4 * T * V - 4), dict(loss=DX),
          dict(loss=W + 8), dict(dx=X + 4), dict(dx=X - 4), dict(dx=X, dt=1), dict(dx=X + 4 * (T - 1) * V),
          dict(dx=W - 4 * T * V + 4), dict(row=W + 4 * T - 4), dict(loss=G), dict(dx=I + 4)]


@pytest.mark.parametrize("kw", SHARED + [dict(stats=TE + 4 * T * K - 4)])
def test_distill(kw):
    assert _distill(**kw) == INV


@pytest.mark.parametrize("kw", SHARED + [dict(logp=RO), dict(logp=ST + 4), dict(logp=LO), dict(logp=O), dict(row=A),
                                         dict(stats=R + 4), dict(logp=X + 8), dict(dx=LP - 8)])
def test_policy(kw):
    assert _policy(**kw) == INV


BACK = [dict(dx=X), dict(dx=X + 4), dict(dx=X - 4 * T * V + 4), dict(dx=ST + 4), dict(dx=W + 4 * T - 4), dict(dx=G),
        dict(dx=I - 4 * T * V + 4)]


@pytest.mark.parametrize("kw", BACK + [dict(dx=TE + 4)])
def test_distill_backward(kw):
    assert _distill_bwd(**kw) == INV


@pytest.mark.parametrize("kw", BACK + [dict(dx=O + 4), dict(dx=A + 4), dict(dx=R + 4)])
def test_policy_backward(kw):
    assert _policy_bwd(**kw) == INV


@pytest.mark.parametrize("kw", [dict(logp=ST), dict(logp=ST + 8 * T - 4), dict(stats=LP + 4), dict(logp=X + 4),
                                dict(stats=I + 4)])
def test_token_logp(kw):
    assert _logp(**kw) == INV


@pytest.mark.parametrize("out", [X + 128, X + 4 * V * D - 4, X - 4 * T * D + 4, I + 4 * T - 4])
def test_embedding(out):
    assert L.moe_embedding(T, V, D, I, X, 0, 1.0, out, 0, None) == INV


@pytest.mark.parametrize("kw", [dict(table=X + 4), dict(table=X - 4 * V * D + 4), dict(table=I + 4), dict(ws=X),
                                dict(ws=DX + 256), dict(ws=I)])
def test_embedding_backward(kw):
    a = dict(table=DX, ws=W) | kw
    assert L.moe_embedding_backward(T, V, D, I, X, 0, 1.0, a["table"], 0, 0, a["ws"], 1 << 20, None) == INV
