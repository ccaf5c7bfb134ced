"""TokenModel keeps what it needs of a batch: a loader may refill its buffers between
forward and backward."""
import pytest
import torch

import moe_expert_routing_sqrt_amd as M

from gpu_util import need_gpu
from test_gpu_token_model import T, _batch, _model

pytestmark = pytest.mark.gpu


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
