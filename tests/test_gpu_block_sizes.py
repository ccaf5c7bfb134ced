"""MoEBlock refuses inputs that are not its layer's size."""
import pytest
import torch

import moe_expert_routing_sqrt_amd as M

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

T, D, E, G, MG, K, FF = 192, 256, 16, 4, 2, 2, 256


def _block(dev):
    g = torch.Generator(device=dev).manual_seed(2)
    w = lambda *s: (0.05 * torch.randn(*s, generator=g, device=dev)).to(torch.bfloat16)  # noqa: E731
    layer = M.MoELayer(T, D, E, G, MG, K, FF, "bf16", 0.05 * torch.randn(D, E, generator=g, device=dev),
                       torch.zeros(E, device=dev), w(E, 2 * FF, D), w(E, D, FF))
    act = lambda: torch.randn(T, D, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    return M.MoEBlock(layer, torch.ones(D, device=dev), torch.zeros(D, device=dev), alpha=1.0), act(), act()


def test_block_refuses_other_sizes():
    """Fewer rows than the layer's would leave the rest of its input as it was."""
    dev = need_gpu()
    blk, delta, stream = _block(dev)
    for a, b in ((delta[:100], stream[:100]), (delta[:100], stream), (delta, stream[:100]),
                 (delta, torch.cat([stream, stream])), (torch.cat([delta, delta]), torch.cat([stream, stream]))):
        with pytest.raises(ValueError):
            blk.forward(a, b)
    blk.forward(delta, stream)
    for bad in (dict(d_out=delta[:100]), dict(d_out=torch.cat([delta, delta])), dict(d_out=delta, d_stream=stream[:100]),
                dict(d_out=delta, d_stream=torch.cat([stream, stream]))):
        with pytest.raises(ValueError):
            blk.backward(**bad)
