"""TokenModel keeps what it needs of a batch: a loader may refill its buffers between
forward and backward.  Its optimizer's masters are its own.  The tied table's gradient is
held in fp32."""
import numpy as np
import pytest
import torch

import moe_expert_routing_sqrt_amd as M
from oracle import embedding as OE

from gpu_util import host, need_gpu
from test_gpu_token_model import D, T, V, _batch, _model

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _run(m, ids, pos, batch, refill=False):
    idx, t, w = batch
    logits = m.forward(ids, pos)
    if refill:
        ids.fill_(3)
        pos.fill_(T - 1)
    m.backward(M.distill_loss(logits, idx, t, weight=w, dlogits=logits)[3])
    return m.d_table.clone(), m.d_positions.clone()


def test_refilled_ids():
    dev = need_gpu()
    m, ids, pos, g = _model(dev)
    batch = _batch(g, dev, ids)
    want = _run(m, ids, pos, batch)
    got = _run(m, ids.clone(), pos.clone(), batch, refill=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_a_block_with_masters_of_its_own():
    dev = need_gpu()
    m, ids, pos, g = _model(dev)
    blk = m.block
    blk.master = [None, None] + [w.float() if w.dtype is torch.bfloat16 else None
                                 for w in (blk.layer.w_gate, blk.layer.w13, blk.layer.w2, blk.layer.sh_w13,
                                           blk.layer.sh_w2)]
    _run(m, ids, pos, _batch(g, dev, ids))
    before = m.table.clone()
    m.step()
    assert not torch.equal(before, m.table) and torch.equal(m.table, m.opt.master[0].to(torch.bfloat16))
    kept = [m.table.float() * 1.001, None, None, None]
    m2 = M.TokenModel(blk, m.table, m.positions, m.norm_w, m.norm_b, scale=7.0, master=kept)
    _run(m2, ids, pos, _batch(g, dev, ids))
    m2.step()
    assert m2.opt.master[0] is kept[0] and torch.equal(m2.table, kept[0].to(torch.bfloat16))


def test_the_tables_gradient_is_fp32():
    """Head and lookup are added in fp32: the head's sums have at most T + 1 roundings on a
    term's way, the lookup's n + 1, and the sum of both one more."""
    dev = need_gpu()
    m, ids, pos, g = _model(dev)
    idx, t, w = _batch(g, dev, ids)
    logits = m.forward(ids, pos)
    dx = M.distill_loss(logits, idx, t, weight=w, dlogits=logits)[3]
    dl = dx.clone()
    m.backward(dx)
    assert m.d_table.dtype is torch.float32
    a, b = host(dl).astype(np.float64), host(m.y).astype(np.float64)
    look, mags, n = OE.backward(host(m.block.dx), host(ids), V, 7.0)
    ref = a.T @ b + look
    tol = U * ((T + 1) * (np.abs(a).T @ np.abs(b)) + (n[:, None] + 1) * mags + 2 * np.abs(ref))
    assert m.d_table.shape == (V, D) and (np.abs(host(m.d_table) - ref) <= tol + 1e-30).all()
