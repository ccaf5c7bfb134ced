"""Refusals of the training-step calls (no GPU: every case fails its host-side
check, or has nothing to launch) and their struct layouts."""
import ctypes

import pytest
import torch

import moe_expert_routing_sqrt_amd as M
from moe_expert_routing_sqrt_amd import _lib

L = _lib.load()
FAKE = 0x1000
INV, UNS, WS = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")


def _norm(rows=4, d=8, x=FAKE, r=None, xt=1, w=FAKE, b=None, eps=1e-5, s=None, y=FAKE, yt=1, mean=FAKE, rstd=FAKE):
    return L.moe_layer_norm(rows, d, x, r, xt, w, b, eps, s, y, yt, mean, rstd, None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INV), (dict(d=0), INV), (dict(x=None), INV), (dict(w=None), INV), (dict(y=None), INV),
    (dict(xt=2), INV), (dict(yt=7), INV), (dict(eps=-1e-9), INV), (dict(eps=NAN), INV), (dict(eps=INF), INV),
    (dict(r=FAKE), INV), (dict(s=FAKE), INV), (dict(mean=None), INV), (dict(rstd=None), INV),
    (dict(xt=0), INV), (dict(x=0x2000, r=FAKE, s=0x3000, xt=0), INV), (dict(x=0x2000, r=0x3000, s=FAKE), INV),
    (dict(d=32769), UNS), (dict(rows=2 ** 31), UNS), (dict(rows=0, x=None, y=None), 0)])
def test_layer_norm_refusals(kw, want):
    assert _norm(**kw) == want


DY, X = 0x2000, 0x3000


def _norm_bwd(rows=1000, d=8, dy=DY, dt=1, x=X, xt=1, w=FAKE, mean=FAKE, rstd=FAKE, ds=None, dx=FAKE, ot=1,
              dw=FAKE, db=None, ws=FAKE, n=1 << 30):
    return L.moe_layer_norm_backward(rows, d, dy, dt, x, xt, w, mean, rstd, ds, dx, ot, dw, db, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INV), (dict(d=-3), INV), (dict(dy=None), INV), (dict(x=None), INV), (dict(w=None), INV),
    (dict(mean=None), INV), (dict(rstd=None), INV), (dict(dx=None), INV), (dict(dw=None), INV), (dict(dt=2), INV),
    (dict(xt=-1), INV), (dict(ot=3), INV), (dict(dx=DY), INV), (dict(dx=X), INV), (dict(ds=FAKE, ot=0), INV),
    (dict(d=40000), UNS), (dict(ws=None), WS), (dict(ws=FAKE + 8), WS), (dict(rows=0, dw=None), INV)])
def test_layer_norm_backward_refusals(kw, want):
    assert _norm_bwd(**kw) == want


def test_layer_norm_backward_workspace():
    for rows, d in ((1000, 1), (500, 8), (1000, 1001), (16384, 7168), (600, 16384)):
        sh = _lib.MoeShape(rows, d, 1, 1, 1, 1, 1, 1)
        need = L.moe_workspace_size(_lib.MOE_OP_LAYER_NORM_BACKWARD, ctypes.byref(sh), 0)
        assert need >= 2 * d * 4
        assert _norm_bwd(rows=rows, d=d, n=need - 1) == WS
    for rows, d in ((8, 7168), (2000, 20000)):       # one launch forms everything: no parts
        few = _lib.MoeShape(rows, d, 1, 1, 1, 1, 1, 1)
        assert L.moe_workspace_size(_lib.MOE_OP_LAYER_NORM_BACKWARD, ctypes.byref(few), 0) == 0
    bad = _lib.MoeShape(1, 40000, 1, 1, 1, 1, 1, 1)
    assert L.moe_workspace_size(_lib.MOE_OP_LAYER_NORM_BACKWARD, ctypes.byref(bad), 0) == 0


def _sh(T=16, E=16, k=4):
    return _lib.MoeShape(T, 1, E, 1, 1, k, 1, 1)


def _loss(sh=None, logits=FAKE, idx=FAKE, off=FAKE, n=2, alpha=0.1, counts=FAKE, prob=FAKE, dprob=FAKE, loss=FAKE,
          ws=FAKE, size=1 << 30):
    sh = _sh(T=1000) if sh is None else sh
    return L.moe_balance_loss(ctypes.byref(sh), logits, None, idx, off, n, None, alpha, counts, prob, dprob, loss, ws,
                              size, None)


@pytest.mark.parametrize("kw,want", [
    (dict(sh=_sh(T=-1)), INV), (dict(sh=_sh(E=0)), INV), (dict(sh=_sh(k=0)), INV), (dict(sh=_sh(k=17)), INV),
    (dict(sh=_sh(E=64, k=17)), UNS), (dict(sh=_sh(E=1025)), UNS), (dict(n=0), INV), (dict(n=65536), UNS),
    (dict(sh=_sh(T=2 ** 31)), UNS), (dict(sh=_sh(T=2 ** 26)), UNS), (dict(off=None), INV), (dict(alpha=NAN), INV),
    (dict(alpha=INF), INV),
    (dict(logits=None), INV), (dict(idx=None), INV), (dict(counts=None), INV), (dict(prob=None), INV),
    (dict(dprob=None), INV), (dict(loss=None), INV), (dict(ws=None), WS), (dict(ws=FAKE + 128), WS)])
def test_balance_loss_refusals(kw, want):
    assert _loss(**kw) == want


def test_balance_loss_workspace():
    for T, E, n in ((65, 8, 1), (0, 512, 1), (10, 256, 40), (5000, 256, 7)):
        sh = _sh(T, E)
        need = L.moe_balance_loss_workspace_size(ctypes.byref(sh), n)
        assert need > 0 and _loss(sh=sh, n=n, size=need - 1) == WS
    for T, E, n in ((0, 8, 1), (64, 256, 32), (1, 1, 1024)):  # one launch, no parts
        assert L.moe_balance_loss_workspace_size(ctypes.byref(_sh(T, E, 1)), n) == 0
    assert L.moe_balance_loss_workspace_size(ctypes.byref(_sh()), 0) == 0
    assert L.moe_balance_loss_workspace_size(None, 1) == 0


def _loss_bwd(sh=None, logits=FAKE, off=FAKE, n=2, dprob=FAKE, dl=FAKE):
    sh = _sh() if sh is None else sh
    return L.moe_balance_loss_backward(ctypes.byref(sh), logits, None, off, n, None, dprob, None, None, dl, None)


@pytest.mark.parametrize("kw,want", [
    (dict(sh=_sh(k=99)), INV), (dict(sh=_sh(E=2000)), UNS), (dict(off=None), INV), (dict(n=-1), INV),
    (dict(logits=None), INV), (dict(dprob=None), INV), (dict(dl=None), INV), (dict(sh=_sh(T=0), logits=None), 0)])
def test_balance_loss_backward_refusals(kw, want):
    assert _loss_bwd(**kw) == want


def test_route_backward_add_refuses_like_the_plain_call():
    sh = _lib.MoeShape(16, 64, 16, 4, 2, 4, 2, 32)
    for fn in (L.moe_route_backward, L.moe_route_backward_add):
        def call(x=FAKE, dt=1, dl=FAKE, ws=FAKE):
            return fn(ctypes.byref(sh), x, dt, FAKE, None, FAKE, FAKE, FAKE, dl, FAKE, FAKE, ws, 1 << 30, None)
        assert call(x=None) == INV and call(dt=2) == INV and call(dl=None) == INV


def _adam(n=1, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, step=1, tensors=True, params=True, **kw):
    f = dict(n=8, param=FAKE, grad=FAKE, master=None, m=FAKE, v=FAKE, m_scale=None, v_scale=None, weight_decay=0.0,
             param_dtype=0, grad_dtype=0, state_dtype=0)
    f.update(kw)
    t = _lib.MoeAdamwTensor(**f)
    h = _lib.MoeAdamwParams(lr, b1, b2, eps, step)
    return L.moe_adamw_step(n, ctypes.byref(t) if tensors else None, ctypes.byref(h) if params else None, None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(params=False), INV), (dict(tensors=False), INV), (dict(lr=-1.0), INV), (dict(lr=NAN), INV),
    (dict(b1=1.0), INV), (dict(b2=-0.1), INV), (dict(b2=NAN), INV), (dict(eps=0.0), INV), (dict(eps=1e-60), INV),
    (dict(eps=INF), INV), (dict(step=0), INV), (dict(param=None), INV), (dict(grad=None), INV), (dict(m=None), INV),
    (dict(v=None), INV), (dict(param_dtype=2), INV), (dict(grad_dtype=9), INV), (dict(state_dtype=1), INV),
    (dict(state_dtype=2), INV), (dict(state_dtype=2, m_scale=FAKE), INV), (dict(master=FAKE), INV),
    (dict(weight_decay=NAN), INV), (dict(**{"n": -1}), INV)])
def test_adamw_refusals(kw, want):
    assert _adam(**kw) == want


def test_adamw_tensor_refusals_and_nothing_to_do():
    t = _lib.MoeAdamwTensor(n=-1, param_dtype=0)
    h = _lib.MoeAdamwParams(1e-3, 0.9, 0.99, 1e-8, 1)
    assert L.moe_adamw_step(1, ctypes.byref(t), ctypes.byref(h), None, None) == INV
    t = _lib.MoeAdamwTensor(n=2 ** 41, param=FAKE, grad=FAKE, m=FAKE, v=FAKE)
    assert L.moe_adamw_step(1, ctypes.byref(t), ctypes.byref(h), None, None) == UNS
    t = _lib.MoeAdamwTensor(n=0)
    assert L.moe_adamw_step(1, ctypes.byref(t), ctypes.byref(h), None, None) == 0
    assert L.moe_adamw_step(0, None, ctypes.byref(h), None, None) == 0


def test_struct_layout():
    assert ctypes.sizeof(_lib.MoeAdamwTensor) == 8 * 8 + 8 + 4 * 4
    assert _lib.MoeAdamwTensor.weight_decay.offset == 64
    assert ctypes.sizeof(_lib.MoeAdamwParams) == 40


def test_binding_refuses_cpu_tensors_types_and_sizes():
    x = torch.zeros(4, 8)
    w = torch.ones(8)
    with pytest.raises(ValueError):
        M.layer_norm(x, w)                                           # not on the GPU
    with pytest.raises(TypeError):
        M.layer_norm(x, w.double())
    with pytest.raises(ValueError):
        M.layer_norm(x, w[:5])
    with pytest.raises(TypeError):
        M.layer_norm(x, w, residual=x.bfloat16())
    with pytest.raises(ValueError):
        M.layer_norm(x, w, sum_out=x)
    sh = M.shape(4, 1, 8, 1, 1, 2, 1, 1)
    idx = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(TypeError):
        M.balance_loss(sh, x, idx.long(), 0.1)
    with pytest.raises(TypeError):
        M.balance_loss(sh, x, idx, 0.1, seq_offsets=torch.tensor([0, 4]))
    with pytest.raises(TypeError):
        M.balance_loss(sh, x, idx, 0.1, token_mask=torch.ones(4))
    with pytest.raises(ValueError):
        M.balance_loss(sh, x, idx, 0.1, token_mask=torch.ones(3, dtype=torch.bool))
    with pytest.raises(ValueError):
        M.AdamW([w], [], lr=1e-3)
    with pytest.raises(ValueError):
        M.AdamW([w], [w[:4]], lr=1e-3)
    with pytest.raises(ValueError):
        M.AdamW([w], [w], lr=1e-3, states="int4")
    with pytest.raises(ValueError):
        M.route_backward(sh, x, x, x, idx, x, x, add_dlogits=True)
