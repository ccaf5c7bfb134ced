"""GPU parity of the losses on logits where a work-group walks several rows: the
distillation's lists, entries carried ahead and rows that do not count between
counted ones; rows longer than what the registers hold; and more units of the gradient
alone than its launch has work-groups.

A row's results do not depend on its neighbours, so every row is held to the same
row in a call of few rows bit by bit, and those to the fp64 oracle by the tolerances
of test_gpu_vocab_loss.py."""
import numpy as np
import pytest
import torch

import moe_expert_routing_sqrt_amd as M

from gpu_util import need_gpu
from test_gpu_vocab_loss import _check_distill, _check_policy

pytestmark = pytest.mark.gpu


def _case(g, T, V, K, dt, dev):
    """logits, entries (repeats, rows without any, padding), teacher, weights; rows of
    weight 0 hold NaN"""
    x = torch.randn(T, V, generator=g, device=dev).to(dt)
    idx = torch.randint(0, V, (T, K), generator=g, device=dev, dtype=torch.int32)
    if K > 4:
        idx[::3, 1], idx[1::5, 4] = idx[::3, 0], idx[1::5, 2]
        idx[2::7] = idx[2::7, :1] + torch.arange(K, device=dev, dtype=torch.int32) % 5  # some past V - 1
    idx[4::11] = -1
    t = 2 * torch.randn(T, K, generator=g, device=dev)
    t[5::13, 0] = float("-inf")
    w = torch.rand(T, generator=g, device=dev) * (torch.rand(T, generator=g, device=dev) > 0.3)
    x[w == 0] = float("nan")
    return x, idx.contiguous(), t, w


def _walk(T, V, K, dt, dev, check=True):
    print(f"distill rows {T}x{V} K={K} {dt}", flush=True)
    g = torch.Generator(device=dev).manual_seed(T + V + K)
    x, idx, t, w = _case(g, T, V, K, dt, dev)
    got = M.distill_loss(x, idx, t, 1.3, w, with_grad=True)
    rows = torch.cat([torch.arange(12), torch.randint(0, T, (20,)), torch.tensor([T - 2, T - 1])]).to(dev)
    part = tuple(a[rows].contiguous() for a in (x, idx, t, w))
    sub = M.distill_loss(*part[:3], 1.3, part[3], with_grad=True)
    for a, b in zip(sub[1:], got[1:]):
        assert torch.equal(a, b[rows])
    live = part[3] != 0
    if check and V < 50000:
        few = tuple(a[live][:12].contiguous() for a in part)
        _check_distill(few[0], few[1], few[2], 1.3, few[3], 1.0, None, sub[3][live][:12],
                       "bf16" if dt is torch.bfloat16 else "f32")
    assert not got[3][w == 0].any() and not got[2][w == 0].any() and not got[1][w == 0].any()
    for _ in range(2):
        again = M.distill_loss(x, idx, t, 1.3, w, with_grad=True)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
    del again
    alone = M.distill_loss(x, idx, t, 1.3, w)
    assert all(torch.equal(a, b) for a, b in zip(got[:3], alone[:3]))
    assert torch.equal(M.distill_loss_backward(x, got[2], idx, t, 1.3, w), got[3])
    total = (w.double() * got[1].double())[w != 0].sum()
    assert abs(float(got[0]) - float(total)) <= 2 ** -23 * abs(float(total)) + 1e-12 * float((w * got[1].abs()).sum())
    over = M.distill_loss(x, idx, t, 1.3, w, dlogits=x)
    assert over[3] is x and all(torch.equal(a, b) for a, b in zip(got, over))


@pytest.mark.parametrize("K", [5, 65, 256])
@pytest.mark.parametrize("T,V", [(20001, 40), (9001, 1500), (4003, 5000), (5001, 9000), (3001, 12300), (2501, 17000),
                                 (2001, 30000), (1101, 40000), (1201, 65000), (601, 90000), (701, 131072)])
def test_distill_rows(T, V, K):
    _walk(T, V, K, torch.bfloat16, need_gpu())


@pytest.mark.parametrize("K", [5, 256])
@pytest.mark.parametrize("T,V", [(9001, 1001), (2501, 9001), (801, 40001)])
def test_distill_rows_fp32(T, V, K):
    _walk(T, V, K, torch.float32, need_gpu())


@pytest.mark.parametrize("K", [5, 256])
def test_distill_rows_past_the_registers(K):
    _walk(601, 140003, K, torch.bfloat16, need_gpu())
    _walk(520, 70001, K, torch.float32, need_gpu())


@pytest.mark.parametrize("T,V,dt", [(601, 140003, torch.bfloat16), (520, 70001, torch.float32)])
def test_policy_rows_past_the_registers(T, V, dt):
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(T)
    x = torch.randn(T, V, generator=g, device=dev).to(dt)
    tok = torch.randint(-V // 9, V, (T,), generator=g, device=dev, dtype=torch.int32)
    w = (torch.rand(T, generator=g, device=dev) > 0.3).float()
    x[w == 0] = float("nan")
    old, adv = torch.full((T,), -float(np.log(V)), device=dev), torch.randn(T, generator=g, device=dev)
    kw = dict(clip=(0.5, 1.0))
    got = M.policy_loss(x, tok, old, adv, weight=w, with_grad=True, **kw)
    rows = torch.cat([torch.arange(6), torch.randint(0, T, (10,)), torch.tensor([T - 1])]).to(dev)
    part = tuple(a[rows].contiguous() for a in (x, tok, old, adv, w))
    sub = M.policy_loss(*part[:4], weight=part[4], with_grad=True, **kw)
    assert all(torch.equal(a, b[rows]) for a, b in zip(sub[1:], got[1:]))
    few = tuple(a[part[4] != 0][:4].contiguous() for a in part)
    _check_policy(*few[:4], None, (0.5, 1.0), 0.0, 1.0, few[4], 1.0, None, sub[4][part[4] != 0][:4],
                  "bf16" if dt is torch.bfloat16 else "f32")
    assert torch.equal(M.policy_loss_backward(x, got[3], tok, old, adv, weight=w, **kw), got[4])
    over = M.policy_loss(x, tok, old, adv, weight=w, dlogits=x, **kw)
    assert over[4] is x and all(torch.equal(a, b) for a, b in zip(got, over))


@pytest.mark.parametrize("T,V,dt", [(70000, 65536, torch.bfloat16), (4400000, 64, torch.bfloat16)])
def test_gradient_alone_beyond_a_launch(T, V, dt):
    """More than 2^20 work-groups' worth of rows: work-groups take several, of which few count."""
    dev = need_gpu()
    print(f"gradient alone {T}x{V}", flush=True)
    g = torch.Generator(device=dev).manual_seed(T)
    K = 6
    x = torch.zeros(T, V, dtype=dt, device=dev)
    live = torch.cat([torch.tensor([0, 1, T // 2, T - 2, T - 1]), torch.randint(0, T, (95,))]).unique().to(dev)
    x[live] = torch.randn(len(live), V, generator=g, device=dev).to(dt)
    idx = torch.randint(0, V, (T, K), generator=g, device=dev, dtype=torch.int32)
    idx[:, 3] = idx[:, 0]
    t = torch.randn(T, K, generator=g, device=dev)
    w = torch.zeros(T, device=dev)
    w[live] = torch.rand(len(live), generator=g, device=dev) + 0.5
    part = tuple(a[live].contiguous() for a in (x, idx, t, w))
    want = M.distill_loss(*part[:3], weight=part[3], with_grad=True)
    stats = torch.zeros(T, 2, device=dev)
    stats[live] = want[2]
    dx = torch.full_like(x, 3.0)
    M.distill_loss_backward(x, stats, idx, t, weight=w, dlogits=dx)
    assert torch.equal(dx[live], want[3])
    dx[live] = 0
    assert not dx.any()
    tok = idx[:, 0].contiguous()
    old, adv = torch.full((T,), -5.0, device=dev), torch.ones(T, device=dev)
    pw = M.policy_loss(part[0], tok[live], old[live], adv[live], weight=part[3], clip=(1.0, 1e6), with_grad=True)
    stats[live] = pw[3]
    dx.fill_(3.0)
    M.policy_loss_backward(x, stats, tok, old, adv, weight=w, clip=(1.0, 1e6), dlogits=dx)
    assert torch.equal(dx[live], pw[4])
    dx[live] = 0
    assert not dx.any()
