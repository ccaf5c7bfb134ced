"""TokenModel: embedding, MoEBlock, norm, tied head and a loss run together as a
training step on token ids.  Each stage is held to the oracle on the values that
reached it, within the stage's own roundings; the table's gradient is the head's
product plus the lookup's."""
import numpy as np
import pytest
import torch

import moe_expert_routing_sqrt_amd as M
from oracle import embedding as OE, norm as ON, vocab_loss as OV

from gpu_util import host, need_gpu

pytestmark = pytest.mark.gpu

T, D, E, G, MG, K, FF, V = 384, 256, 16, 4, 2, 4, 256, 1000
HALF = 2.0 ** -8  # a bf16 rounding


def _model(dev, seed=0, **kw):
    g = torch.Generator(device=dev).manual_seed(seed)
    w = lambda *s, scale=0.05: (scale * torch.randn(*s, generator=g, device=dev)).to(torch.bfloat16)  # noqa: E731
    layer = M.MoELayer(T, D, E, G, MG, K, FF, "bf16", 0.05 * torch.randn(D, E, generator=g, device=dev),
                       torch.zeros(E, device=dev), w(E, 2 * FF, D), w(E, D, FF), w(1, 2 * FF, D), w(1, D, FF))
    one = lambda: 1 + 0.1 * torch.randn(D, generator=g, device=dev)  # noqa: E731
    blk = M.MoEBlock(layer, one(), 0.1 * one(), **kw)
    model = M.TokenModel(blk, w(V, D), w(T, D, scale=0.5), one(), 0.1 * one(), scale=7.0)
    ids = torch.randint(-20, V, (T,), generator=g, device=dev, dtype=torch.int32)  # some padding
    return model, ids, torch.arange(T, device=dev, dtype=torch.int32) % 128, g


def _batch(g, dev, ids):
    idx = torch.randint(0, V, (T, 12), generator=g, device=dev, dtype=torch.int32)
    t = 2 * torch.randn(T, 12, generator=g, device=dev)
    w = (ids >= 0).float() / (ids >= 0).sum()
    return idx, t, w


@pytest.mark.parametrize("kind", ["distill", "policy"])
def test_stages_and_gradients(kind):
    dev = need_gpu()
    m, ids, pos, g = _model(dev)
    idx, t, w = _batch(g, dev, ids)
    logits = m.forward(ids, pos)
    assert logits is m.logits and logits.shape == (T, V)
    ref = OE.forward(host(ids), host(m.table), 7.0)
    assert (np.abs(host(m.stream) - ref) <= (HALF + 2.0 ** -24) * np.abs(ref)).all()
    assert torch.equal(m.delta, m.positions[pos.long()])
    blk = m.block
    assert torch.equal(blk.stream, (m.delta.float() + m.stream.float()).to(torch.bfloat16))
    y, _, _ = ON.forward(host(m.sum), host(m.norm_w), host(m.norm_b))
    assert np.abs(host(m.y) - y).max() <= 2 * HALF * np.abs(y).max()
    z = host(m.y).astype(np.float64) @ host(m.table).astype(np.float64).T
    assert np.abs(host(logits) - z).max() <= 2 * HALF * np.abs(z).max()
    x = logits.clone()
    if kind == "distill":
        loss, row, _, dx = M.distill_loss(logits, idx, t, 2.0, w, dlogits=logits)
        ref = OV.distill(host(x), host(idx), host(t), 2.0, host(w))
    else:
        tok = idx[:, 0].contiguous()
        lp, _ = M.token_logp(x, tok)
        old, adv = lp - 0.1, t[:, 0].contiguous()
        loss, row, _, _, dx = M.policy_loss(logits, tok, old, adv, lp + 0.2, kl=0.1, weight=w, dlogits=logits)
        ref = OV.policy(host(x), host(tok), host(old), host(adv), host(lp + 0.2), (0.2, 0.2), 0.1, 1.0, host(w))
    assert dx is logits and abs(float(loss) - ref["loss"]) <= 1e-5 * np.abs(host(w) * ref["row_loss"]).sum()
    assert np.abs(host(dx) - ref["dlogits"]).max() <= 2 * HALF * np.abs(ref["dlogits"]).max()
    assert not dx[ids < 0].any()
    dl = dx.clone()
    m.backward(dx)
    # the norm's input gradient reaches the block's output and its stream
    dy = host(dl).astype(np.float64) @ host(m.table).astype(np.float64)
    want, dw, db = ON.backward(host(m.dy), host(m.sum), host(m.norm_w), host(m.mean), host(m.rstd))
    assert np.abs(host(m.dy) - dy).max() <= 2 * HALF * np.abs(dy).max()
    assert np.abs(host(m.dx) - want).max() <= 2 * HALF * np.abs(want).max()
    assert np.abs(host(m.d_norm_w) - dw).max() <= 1e-4 * np.abs(dw).max()
    # tied table: head + lookup (two bf16 roundings: the product's, the sum's)
    head = host(dl).astype(np.float64).T @ host(m.y).astype(np.float64)
    look = OE.backward(host(blk.dx), host(ids), V, 7.0)[0]
    err = np.abs(host(m.d_table) - (head + look))
    assert (err <= 2 * HALF * (np.abs(head) + np.abs(look)).max(1, keepdims=True) + 1e-12).all()
    posg = OE.backward(host(blk.dx), host(pos), T)
    assert (np.abs(host(m.d_positions) - posg[0]) <= (posg[2][:, None] + 1) * 2.0 ** -24 * posg[1]).all()
    assert not m.d_positions[128:].any()


def test_steps_change_every_weight_and_a_graph_repeats_them():
    """Three steps move the table, the positions, both norms and the experts; forward,
    loss and backward captured into a graph give the same gradients."""
    dev = need_gpu()
    m, ids, pos, g = _model(dev, 1, lr=1e-3, states="e4m3")
    idx, t, w = _batch(g, dev, ids)
    before = [p.clone() for p in (m.table, m.positions, m.norm_w, m.block.norm_w, m.block.layer.w13)]
    loss = torch.empty(1, device=dev)
    row, stats = torch.empty(T, device=dev), torch.empty(2 * T, device=dev)

    def work():
        lg = m.forward(ids, pos)
        M.distill_loss(lg, idx, t, 1.0, w, loss=loss, row_loss=row, stats=stats, dlogits=lg)
        m.backward(lg)

    for _ in range(3):
        work()
        assert torch.isfinite(loss).all()
        m.step()
    for old, p in zip(before, (m.table, m.positions, m.norm_w, m.block.norm_w, m.block.layer.w13)):
        assert torch.isfinite(p.float()).all() and not torch.equal(old, p)
    assert torch.equal(m.table, m.opt.master[0].to(torch.bfloat16))
    work()
    torch.cuda.synchronize()
    want = [x.clone() for x in (loss, m.d_table, m.d_positions, m.d_norm_w, m.block.grads["dw13"])]
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        work()
    for _ in range(3):
        m.d_table.zero_()
        m.d_positions.fill_(3.0)
        gr.replay()
        torch.cuda.synchronize()
        got = (loss, m.d_table, m.d_positions, m.d_norm_w, m.block.grads["dw13"])
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_refusals():
    dev = need_gpu()
    m, ids, pos, _ = _model(dev)
    with pytest.raises(ValueError, match="ids: needs"):
        m.forward(ids[:-1], pos)
    with pytest.raises(TypeError, match="ids must be int32"):
        m.forward(ids.long(), pos)
    with pytest.raises(ValueError, match="rows of"):
        M.TokenModel(m.block, m.table[:, :-1].contiguous(), m.positions, m.norm_w, m.norm_b)
    m.forward(ids, pos)
    with pytest.raises(ValueError, match="dlogits"):
        m.backward(m.logits.float())


@pytest.mark.parametrize("loss", ["distill", "policy"])
def test_train_step_command(loss, capsys):
    need_gpu()
    from moe_expert_routing_sqrt_amd import train_step
    r = train_step.main(["--workload", "flash", "--tokens", "512", "--steps", "3", "--loss", loss, "--vocab", "5000"])
    assert len(r["errors"]) == 3 and all(np.isfinite(e[0]) for e in r["errors"])
    assert all(v > 0 for v in r["ms"].values())
    assert loss.replace("distill", "distillation") + " loss" in capsys.readouterr().out
