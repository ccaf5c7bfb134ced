"""MoEBlock: norm, MoE layer, balance loss and AdamW run together as a training
step."""
import numpy as np
import pytest
import torch

import moe_expert_routing_sqrt_amd as M
from oracle import adamw as OA, balance_loss as OL, norm as ON

from gpu_util import host, need_gpu

pytestmark = pytest.mark.gpu

T, D, E, G, MG, K, FF = 384, 256, 16, 4, 2, 4, 256


def _block(dev, seed=0, **kw):
    g = torch.Generator(device=dev).manual_seed(seed)
    w = lambda *s, scale=0.05: (scale * torch.randn(*s, generator=g, device=dev)).to(torch.bfloat16)  # noqa: E731
    layer = M.MoELayer(T, D, E, G, MG, K, FF, "bf16", 0.05 * torch.randn(D, E, generator=g, device=dev),
                       torch.zeros(E, device=dev), w(E, 2 * FF, D), w(E, D, FF), w(1, 2 * FF, D), w(1, D, FF))
    nw = 1 + 0.1 * torch.randn(D, generator=g, device=dev)
    return M.MoEBlock(layer, nw, 0.1 * torch.randn(D, generator=g, device=dev), **kw), g


def _acts(g, dev, scale=1.0):
    return (scale * torch.randn(T, D, generator=g, device=dev)).to(torch.bfloat16)


def test_forward_and_backward_pieces():
    dev = need_gpu()
    blk, g = _block(dev, alpha=0.5)
    la = blk.layer
    delta, stream, dout, dst = _acts(g, dev), _acts(g, dev), _acts(g, dev, 0.1), _acts(g, dev, 0.1)
    off = torch.tensor([0, 100, 100, 380], dtype=torch.int32, device=dev)
    mask = torch.rand(T, generator=g, device=dev) > 0.2
    out, s = blk.forward(delta, stream, off, mask)
    out = out.clone()
    assert torch.equal(s, (delta.float() + stream.float()).to(torch.bfloat16))
    # the layer ran on the norm of the new stream; the loss is on its router
    y, mean, rstd = ON.forward(host(s), host(blk.norm_w), host(blk.norm_b))
    assert np.abs(host(blk.h) - y).max() <= 2.0 ** -8 * np.abs(y).max()
    assert torch.equal(la.forward(blk.h, save_for_backward=True), out)
    ref = OL.forward(host(la.logits), host(la.idx), 0.5, host(off), host(mask))
    assert np.array_equal(host(blk.counts), ref[1]) and abs(float(blk.loss) - ref[0]) <= 1e-5 * ref[0]
    dx = blk.backward(dout, dst).clone()
    grads = {k: v.clone() for k, v in blk.grads.items()}
    # by hand: the loss's gradient, the layer's backward with it, the norm's
    dl = M.balance_loss_backward(la.sh, la.logits, blk.dprob, off, mask)
    la._bwd_ws(dev)["dlogits"].copy_(dl)
    by_hand = la.backward(blk.h, dout, add_dlogits=True)
    assert all(torch.equal(by_hand[k], grads[k]) for k in grads)
    want, dw, db = M.layer_norm_backward(grads["dx"], s, blk.norm_w, blk.mean, blk.rstd, d_sum=dst)
    assert torch.equal(dx, want) and torch.equal(blk.d_norm_w, dw) and torch.equal(blk.d_norm_b, db)
    # with no gradient of the output only the balance loss moves the router
    blk.backward(torch.zeros_like(dout))
    hl = OL.backward(host(la.logits), host(blk.dprob), host(off), host(mask))
    rw = host(blk.h).astype(np.float64).T @ hl
    assert np.abs(host(blk.grads["dw_gate"]) - rw).max() <= 1e-4 * np.abs(rw).max()
    assert not blk.grads["dw13"].any()


def test_layer_backward_is_unchanged_without_other_gradients():
    dev = need_gpu()
    blk, g = _block(dev, 3)
    x, gr = _acts(g, dev), _acts(g, dev)
    la = blk.layer
    la.forward(x, save_for_backward=True)
    a = {k: v.clone() for k, v in la.backward(x, gr).items()}
    la._bwd_ws(dev)["dlogits"].fill_(float("nan"))
    b = la.backward(x, gr)
    assert all(torch.equal(a[k], b[k]) for k in a)
    la._bwd_ws(dev)["dlogits"].zero_()
    c = la.backward(x, gr, add_dlogits=True)
    assert all(torch.equal(a[k], c[k]) for k in a)


@pytest.mark.parametrize("states", ["f32", "e4m3"])
def test_training_lowers_the_loss(states):
    """Ten steps towards a fixed target: the squared error falls, every weight is
    its master's rounding, and the first step is the oracle's."""
    dev = need_gpu()
    blk, g = _block(dev, 1, lr=3e-3, states=states)
    la = blk.layer
    delta, stream, target = _acts(g, dev), _acts(g, dev), _acts(g, dev, 0.5)
    errs = []
    w0, nw0 = la.w_gate.clone(), blk.norm_w.clone()
    for i in range(10):
        out, s = blk.forward(delta, stream)
        diff = out.float() - target.float()
        errs.append(float((diff * diff).mean()))
        blk.backward((2 * diff / diff.numel() * 1024).to(torch.bfloat16))
        blk.step(torch.full((1,), 1 / 1024, device=dev))
        if i == 0:
            for w, p, gr, wd in ((w0, la.w_gate, blk.grads["dw_gate"], 0.1), (nw0, blk.norm_w, blk.d_norm_w, 0.0)):
                ref = OA.step(host(w).ravel(), host(gr).ravel(), np.zeros(w.numel()), np.zeros(w.numel()), lr=3e-3,
                              b1=0.9, b2=0.95, eps=1e-8, wd=wd, t=1, scale=1 / 1024)[0]
                assert np.array_equal(host(p).ravel(), ref)
    assert errs[-1] < 0.7 * errs[0], errs
    for p, m in zip(blk.opt.params, blk.opt.master):
        assert m is None or torch.equal(p, m.to(torch.bfloat16))
    assert blk.opt.step_count == 10


def test_train_step_command(capsys):
    need_gpu()
    from moe_expert_routing_sqrt_amd import train_step
    r = train_step.main(["--workload", "flash", "--tokens", "512", "--steps", "4", "--states", "e4m3"])
    assert len(r["errors"]) == 4 and r["errors"][-1][0] < r["errors"][0][0]
    assert all(t > 0 for t in r["ms"].values())
    assert "squared error" in capsys.readouterr().out
