"""Arguments of the token calls whose sizes do not belong together are refused: a larger
buffer would be read in rows of another width, or beside other rows."""
import pytest
import torch

import moe_expert_routing_sqrt_amd as M

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def _batch(dev):
    """A batch of 2 sequences of 5 tokens, the last of each without a next one"""
    g = torch.Generator(device=dev).manual_seed(0)
    logits = torch.randn(2, 5, 40, generator=g, device=dev)[:, :-1].contiguous()
    tok = torch.randint(0, 40, (2, 5), generator=g, device=dev, dtype=torch.int32)
    return logits, tok, torch.randn(2, 5, generator=g, device=dev)


def test_distill_refuses_other_shapes():
    dev = need_gpu()
    x = torch.randn(8, 40, device=dev)
    idx, t = torch.zeros(8, 4, dtype=torch.int32, device=dev), torch.zeros(8, 4, device=dev)
    stats = M.distill_loss(x, idx, t)[2]
    wide, more = torch.zeros(8, 8, device=dev), torch.zeros(9, 4, device=dev)
    for bad in (wide, more, torch.zeros(4, 8, device=dev), t.view(-1)):
        with pytest.raises(ValueError, match="teacher"):
            M.distill_loss(x, idx, bad)
        with pytest.raises(ValueError, match="teacher"):
            M.distill_loss_backward(x, stats, idx, bad)
    with pytest.raises(ValueError, match="idx: needs"):
        M.distill_loss(x[:4], idx, t[:4])
    with pytest.raises(ValueError, match="weight: needs"):
        M.distill_loss(x, idx, t, weight=torch.ones(10, device=dev))
    with pytest.raises(ValueError, match="stats: needs"):
        M.distill_loss_backward(x, torch.zeros(9, 2, device=dev), idx, t)
    with pytest.raises(ValueError, match="grad_loss: needs"):
        M.distill_loss(x, idx, t, grad_loss=torch.ones(2, device=dev), with_grad=True)
    with pytest.raises(ValueError, match="dlogits: needs"):
        M.distill_loss(x[:4], idx[:4], t[:4], dlogits=x)
    with pytest.raises(ValueError, match="row_loss: needs"):
        M.distill_loss(x, idx, t, row_loss=torch.zeros(9, device=dev))


def test_policy_refuses_rows_of_another_batch():
    dev = need_gpu()
    x, tok, f = _batch(dev)
    k, v = tok[:, 1:].contiguous(), f[:, 1:].contiguous()
    ok = M.policy_loss(x, k, v, v, ref_logp=v, kl=0.1, weight=v)
    for name, args, kw in (("tokens", (tok, v, v), {}), ("old_logp", (k, f, v), {}), ("advantage", (k, v, f), {}),
                           ("ref_logp", (k, v, v), dict(ref_logp=f, kl=0.1)), ("weight", (k, v, v), dict(weight=f))):
        with pytest.raises(ValueError, match=f"{name}: needs"):
            M.policy_loss(x, *args, **kw)
        with pytest.raises(ValueError, match=f"{name}: needs"):
            M.policy_loss_backward(x, ok[3], *args, **kw)
    with pytest.raises(ValueError, match="tokens: needs"):
        M.token_logp(x, tok)
    with pytest.raises(ValueError, match="logp: needs"):
        M.token_logp(x, k, logp=torch.zeros(10, device=dev))


def test_embedding_refuses_other_sizes():
    dev = need_gpu()
    ids, table = torch.zeros(6, dtype=torch.int32, device=dev), torch.randn(9, 16, device=dev)
    with pytest.raises(ValueError, match="out: needs"):
        M.embedding(ids, table, out=torch.zeros(7, 16, device=dev))
    with pytest.raises(ValueError, match="d_out: needs"):
        M.embedding_backward(torch.zeros(7, 16, device=dev), ids, 9)
    with pytest.raises(ValueError, match="d_table: needs"):
        M.embedding_backward(torch.zeros(6, 16, device=dev), ids, 8, d_table=table)
