"""MoEBlock with a scaled loss: the balance gradient carries the scale that d_out
does, so that step()'s grad_scale takes it off both."""
import numpy as np
import torch
import pytest

import moe_expert_routing_sqrt_amd as M
from oracle import balance_loss as OL

from gpu_util import host, need_gpu

pytestmark = pytest.mark.gpu

T, D, E, G, MG, K, FF = 320, 256, 16, 4, 2, 4, 256


def _block(dev, **kw):
    g = torch.Generator(device=dev).manual_seed(5)
    w = lambda *s: (0.05 * torch.randn(*s, generator=g, device=dev)).to(torch.bfloat16)  # noqa: E731
    layer = M.MoELayer(T, D, E, G, MG, K, FF, "bf16", 0.05 * torch.randn(D, E, generator=g, device=dev),
                       torch.zeros(E, device=dev), w(E, 2 * FF, D), w(E, D, FF), w(1, 2 * FF, D), w(1, D, FF))
    return M.MoEBlock(layer, torch.ones(D, device=dev), torch.zeros(D, device=dev), **kw), g


def _acts(g, dev, scale=1.0):
    return (scale * torch.randn(T, D, generator=g, device=dev)).to(torch.bfloat16)


def test_scaled_loss_gives_the_scaled_router_gradient():
    """A power of two scales every product exactly: the router's gradient of the
    scaled step is the unscaled one's times it, and holds the whole of alpha."""
    dev = need_gpu()
    blk, g = _block(dev, alpha=4.0)
    la = blk.layer
    delta, stream, dout = _acts(g, dev), _acts(g, dev), _acts(g, dev, 1e-4)
    blk.forward(delta, stream)
    blk.backward(dout)
    one = {k: v.clone() for k, v in blk.grads.items()}
    blk.backward(dout * 1024, grad_loss=torch.full((1,), 1024.0, device=dev))
    for k in ("dw_gate", "dx", "dw13", "dw2"):
        big = one[k].double().abs().max()
        assert (blk.grads[k].double() / 1024 - one[k].double()).abs().max() <= 1e-6 * big, k
    # main + alpha part: the layer's own gradient without a balance loss, and the oracle's
    main = la.backward(blk.h, dout)["dw_gate"]
    dl = OL.backward(host(la.logits), host(blk.dprob))
    part = host(blk.h).astype(np.float64).T @ dl
    want = host(main).astype(np.float64) + part
    assert np.abs(part).max() > 0.1 * np.abs(want).max()          # alpha's part is not lost in the other
    assert np.abs(host(one["dw_gate"]) - want).max() <= 1e-4 * np.abs(want).max()


def test_train_step_scales_both_gradients(monkeypatch):
    need_gpu()
    from moe_expert_routing_sqrt_amd import train_step
    seen = []
    backward, step = M.MoEBlock.backward, M.MoEBlock.step

    def spy_backward(self, d_out, d_stream=None, grad_loss=None):
        seen.append([grad_loss])
        return backward(self, d_out, d_stream, grad_loss)

    def spy_step(self, grad_scale=None):
        seen[-1].append(grad_scale)
        return step(self, grad_scale)

    monkeypatch.setattr(M.MoEBlock, "backward", spy_backward)
    monkeypatch.setattr(M.MoEBlock, "step", spy_step)
    train_step.main(["--workload", "flash", "--tokens", "512", "--steps", "2"])
    assert len(seen) == 2
    for grad_loss, grad_scale in seen:
        assert grad_loss is not None and float(grad_loss) * float(grad_scale) == 1.0
