"""Refusals of the embedding and vocabulary-loss calls (no GPU: every case fails
its host-side check, or has nothing to launch), and of their binding."""
import ctypes

import pytest
import torch

import moe_expert_routing_sqrt_amd as M
from moe_expert_routing_sqrt_amd import _lib

L = _lib.load()
A, B, C, D = 0x1000, 0x2000, 0x3000, 0x4000  # never dereferenced
INV, UNS, WS = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")

SIZES = [(dict(T=-1), INV), (dict(V=0), INV), (dict(V=(1 << 24) + 1), UNS), (dict(T=1 << 26), UNS)]


def _embed(T=4, V=8, d=8, ids=A, table=B, tt=1, scale=1.0, out=C, ot=1):
    return L.moe_embedding(T, V, d, ids, table, tt, scale, out, ot, None)


@pytest.mark.parametrize("kw,want", SIZES + [
    (dict(d=0), INV), (dict(ids=None), INV), (dict(table=None), INV), (dict(out=None), INV), (dict(out=B), INV),
    (dict(tt=2), INV), (dict(ot=-1), INV), (dict(scale=NAN), INV), (dict(scale=INF), INV), (dict(out=A), INV),
    (dict(d=(1 << 20) + 1), UNS),
    (dict(T=0, ids=None, table=None, out=None), 0)])
def test_embedding_refusals(kw, want):
    assert _embed(**kw) == want


def _embed_bwd(T=4, V=8, d=8, ids=A, dy=B, yt=1, scale=1.0, table=C, tt=0, add=0, ws=D, n=1 << 40):
    return L.moe_embedding_backward(T, V, d, ids, dy, yt, scale, table, tt, add, ws, n, None)


@pytest.mark.parametrize("kw,want", SIZES + [
    (dict(d=0), INV), (dict(ids=None), INV), (dict(dy=None), INV), (dict(table=None), INV), (dict(table=B), INV),
    (dict(yt=2), INV), (dict(tt=9), INV), (dict(scale=NAN), INV), (dict(add=2), INV), (dict(ws=None), WS),
    (dict(ws=D + 16), WS), (dict(T=(1 << 26) - 1, d=2049), UNS),
    (dict(T=1, V=1 << 24, d=9000), UNS), (dict(d=(1 << 20) + 1), UNS), (dict(table=A), INV)])
def test_embedding_backward_refusals(kw, want):
    assert _embed_bwd(**kw) == want


def test_embedding_backward_workspace():
    for T, V, d in ((1, 1, 1), (1000, 5003, 1001), (16384, 131072, 7168), (0, 50, 8)):
        need = L.moe_embedding_backward_workspace_size(T, V, d)
        assert need >= 8 * T + 4 * V
        assert _embed_bwd(T=T, V=V, d=d, n=need - 1) == WS
    for bad in ((-1, 8, 8), (4, 0, 8), (4, 8, 0), (1 << 26, 8, 8), (4, 8, (1 << 20) + 1)):
        assert L.moe_embedding_backward_workspace_size(*bad) == 0


def _distill(T=4, V=8, K=2, x=A, xt=1, idx=B, t=C, tt=0, tau=1.0, w=None, loss=D, row=D, stats=D, dx=None, dt=1):
    return L.moe_distill_loss(T, V, K, x, xt, idx, t, tt, tau, w, None, loss, row, stats, dx, dt, None)


def _distill_bwd(T=4, V=8, K=2, x=A, xt=1, idx=B, t=C, tt=0, tau=1.0, stats=D, dx=0x5000, dt=1):
    return L.moe_distill_loss_backward(T, V, K, x, xt, stats, idx, t, tt, tau, None, None, dx, dt, None)


DISTILL = SIZES + [(dict(K=0), INV), (dict(K=257), UNS), (dict(x=None), INV), (dict(xt=2), INV), (dict(idx=None), INV),
                   (dict(t=None), INV), (dict(tt=5), INV), (dict(tau=0.0), INV), (dict(tau=-1.0), INV),
                   (dict(tau=NAN), INV), (dict(tau=INF), INV), (dict(tau=1e-39), INV), (dict(tau=1e39), INV),
                   (dict(stats=None), INV)]


@pytest.mark.parametrize("kw,want", DISTILL + [
    (dict(loss=None), INV), (dict(row=None), INV), (dict(dx=0x5000, dt=2), INV), (dict(dx=A, dt=0), INV),
    (dict(w=D), INV), (dict(row=C), INV), (dict(stats=A), INV), (dict(dx=D), INV), (dict(dx=C), INV)])
def test_distill_refusals(kw, want):
    assert _distill(**kw) == want


@pytest.mark.parametrize("kw,want", DISTILL + [
    (dict(dx=None), INV), (dict(dt=2), INV), (dict(dx=A), INV), (dict(dx=A, dt=0), INV),
    (dict(dx=B), INV), (dict(dx=C), INV), (dict(dx=D), INV),
    (dict(T=0, x=None, idx=None, t=None, stats=None, dx=None), 0)])
def test_distill_backward_refusals(kw, want):
    assert _distill_bwd(**kw) == want


def _h(tau=1.0, lo=0.2, hi=0.2, kl=0.0):
    return _lib.MoePolicyParams(tau, lo, hi, kl)


def _policy(T=4, V=8, x=A, xt=1, tok=B, old=C, adv=C, ref=None, h=_h(), loss=D, row=D, logp=D, stats=D, dx=None, dt=1):
    return L.moe_policy_loss(T, V, x, xt, tok, old, adv, ref, None if h is None else ctypes.byref(h), None, None, loss,
                             row, logp, stats, dx, dt, None)


def _policy_bwd(T=4, V=8, x=A, xt=1, tok=B, old=C, adv=C, ref=None, h=_h(), stats=D, dx=0x5000, dt=1):
    return L.moe_policy_loss_backward(T, V, x, xt, stats, tok, old, adv, ref, None if h is None else ctypes.byref(h),
                                      None, None, dx, dt, None)


POLICY = SIZES + [(dict(x=None), INV), (dict(xt=2), INV), (dict(tok=None), INV), (dict(old=None), INV),
                  (dict(adv=None), INV), (dict(h=None), INV), (dict(h=_h(tau=0.0)), INV), (dict(h=_h(tau=NAN)), INV),
                  (dict(h=_h(lo=-0.1)), INV), (dict(h=_h(hi=INF)), INV), (dict(h=_h(hi=NAN)), INV),
                  (dict(h=_h(kl=-1.0)), INV), (dict(h=_h(kl=0.1)), INV), (dict(stats=None), INV)]


@pytest.mark.parametrize("kw,want", POLICY + [
    (dict(loss=None), INV), (dict(row=None), INV), (dict(logp=None), INV), (dict(dx=0x5000, dt=7), INV),
    (dict(dx=A, dt=0), INV), (dict(logp=C), INV), (dict(row=C), INV), (dict(stats=A), INV), (dict(dx=D), INV)])
def test_policy_refusals(kw, want):
    assert _policy(**kw) == want


@pytest.mark.parametrize("kw,want", POLICY + [
    (dict(dx=None), INV), (dict(dt=2), INV), (dict(dx=A), INV),
    (dict(dx=B), INV), (dict(dx=C), INV), (dict(dx=D), INV),
    (dict(T=0, x=None, tok=None, old=None, adv=None, stats=None, dx=None), 0)])
def test_policy_backward_refusals(kw, want):
    assert _policy_bwd(**kw) == want


def _logp(T=4, V=8, x=A, xt=1, tok=B, tau=1.0, logp=C, stats=D):
    return L.moe_token_logp(T, V, x, xt, tok, tau, logp, stats, None)


@pytest.mark.parametrize("kw,want", SIZES + [
    (dict(x=None), INV), (dict(xt=2), INV), (dict(tok=None), INV), (dict(tau=0.0), INV), (dict(logp=None), INV),
    (dict(stats=None), INV), (dict(logp=A), INV), (dict(stats=B), INV), (dict(T=0, x=None, tok=None), 0)])
def test_token_logp_refusals(kw, want):
    assert _logp(**kw) == want


def test_policy_params_layout():
    assert ctypes.sizeof(_lib.MoePolicyParams) == 32 and _lib.MoePolicyParams.kl.offset == 24


def test_binding_refuses_before_the_library():
    """Tensors on the CPU, of a wrong type or too small."""
    x, i = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError, match="ids must be int32"):
        M.embedding(i.long(), x)
    with pytest.raises(ValueError, match="GPU"):
        M.embedding(i, x)
    with pytest.raises(ValueError, match="GPU"):
        M.embedding_backward(x, i, 8)
    with pytest.raises(ValueError, match="logits must be"):
        M.distill_loss(x[0], i.view(4, 1), x[:, :1])
    with pytest.raises(ValueError, match="GPU"):
        M.distill_loss(x, i.view(4, 1), x[:, :1].contiguous())
    with pytest.raises(ValueError, match="GPU"):
        M.policy_loss(x, i, x[:, 0].contiguous(), x[:, 0].contiguous())
    with pytest.raises(ValueError, match="GPU"):
        M.token_logp(x, i)

