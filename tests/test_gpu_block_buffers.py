"""MoEBlock's balance-loss buffers over many numbers of sequences."""
import ctypes

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


def _held(blk):
    """Bytes of every tensor that the block holds itself, by storage."""
    found = {}

    def walk(v):
        if isinstance(v, torch.Tensor):
            found[v.untyped_storage().data_ptr()] = v.untyped_storage().nbytes()
        elif isinstance(v, dict):
            for x in v.values():
                walk(x)
        elif isinstance(v, (list, tuple)):
            for x in v:
                walk(x)

    for k, v in vars(blk).items():
        if k not in ("layer", "opt", "seqs"):
            walk(v)
    return sum(found.values())


def test_buffers_of_many_sequence_counts_stay_bounded():
    dev = need_gpu()
    blk, delta, stream = _block(dev)
    most = 150
    off = lambda n: (torch.arange(n + 1, device=dev) * T // n).to(torch.int32)  # noqa: E731
    blk.forward(delta, stream, off(most))
    one = _held(blk)
    ws = M.lib().moe_balance_loss_workspace_size
    # two sets of the largest count's buffers and the blocks' rounding
    table = (3 * most * E * 4 + int(ws(ctypes.byref(blk.layer.sh), most))) * 2 + 64 * 1024
    for n in range(1, most + 1):
        blk.forward(delta, stream, off(n))
        want = M.balance_loss(blk.layer.sh, blk.layer.logits, blk.layer.idx, 1.0, seq_offsets=off(n))
        assert blk.counts.shape == (n, E) and blk.dprob.shape == (n, E)
        assert all(torch.equal(p, q) for p, q in zip((blk.loss, blk.counts, blk.prob, blk.dprob), want)), n
    assert _held(blk) <= one + table, (one, _held(blk))


def test_a_captured_step_stays_valid_after_larger_sequence_counts():
    dev = need_gpu()
    blk, delta, stream = _block(dev)
    off = (torch.arange(4, device=dev) * T // 3).to(torch.int32)
    blk.forward(delta, stream, off)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        blk.forward(delta, stream, off)
    loss, dprob = blk.loss, blk.dprob
    for n in (2, 3, 4, 70, 190):
        blk.forward(delta, stream, (torch.arange(n + 1, device=dev) * T // n).to(torch.int32))
        other = [torch.full((1 << 18,), 7.0, device=dev) for _ in range(8)]   # takes what was freed
        graph.replay()
        torch.cuda.synchronize()
        want = M.balance_loss(blk.layer.sh, blk.layer.logits, blk.layer.idx, 1.0, seq_offsets=off)
        assert torch.equal(loss, want[0]) and torch.equal(dprob, want[3]), n
        assert all(bool((o == 7).all()) for o in other)
