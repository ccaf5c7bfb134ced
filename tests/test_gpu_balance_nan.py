"""A counted token whose logits are not numbers: the balance loss, its sequence's
probabilities and its own gradient are NaN in every form of the call (at most 64
tokens, short sequences, long ones), and nothing else is touched."""
import numpy as np
import pytest
import torch

import moe_expert_routing_sqrt_amd as M
from oracle import balance_loss as OL

from gpu_util import dev_f32, dev_i32, host, need_gpu

pytestmark = pytest.mark.gpu

# T, E, k, sequences: one launch; short sequences; long ones at one, two and four column groups a lane
FORMS = [(40, 64, 4, 5), (33, 7, 2, 3), (300, 64, 4, 40), (200, 31, 3, 33), (900, 64, 4, 5), (130, 30, 3, 1),
         (400, 300, 4, 3), (200, 1000, 2, 2)]


def _case(T, E, k, n):
    rng = np.random.default_rng(T + E)
    L = rng.normal(size=(T, E)).astype(np.float32)
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    return L, idx, (np.arange(n + 1) * T // n).astype(np.int32)


@pytest.mark.parametrize("bad", ["one", "row", "inf"])
@pytest.mark.parametrize("T,E,k,n", FORMS)
def test_counted_nan(T, E, k, n, bad):
    dev = need_gpu()
    print(f"balance loss with {bad} T={T} E={E} k={k} n={n}", flush=True)
    L, idx, off = _case(T, E, k, n)
    sh, id_, kw = M.shape(T, 1, E, 1, 1, k, 1, 1), dev_i32(idx, dev), dict(seq_offsets=dev_i32(off, dev))
    s = n // 2
    t = int(off[s]) + 1
    L2 = L.copy()
    L2[t, slice(None) if bad == "row" else E // 3] = np.inf if bad == "inf" else np.nan
    clean = M.balance_loss(sh, dev_f32(L, dev), id_, 0.1, **kw)
    got = M.balance_loss(sh, dev_f32(L2, dev), id_, 0.1, **kw)
    extra = dev_f32(np.ones((T, E)), dev)
    grads = [[M.balance_loss_backward(sh, dev_f32(x, dev), clean[3], d_extra=e, **kw) for x in (L, L2)]
             for e in (None, extra)]
    torch.cuda.synchronize()
    loss, counts, prob, dprob = got
    assert torch.isnan(loss).all()
    assert torch.equal(counts, clean[1]) and torch.equal(dprob, clean[3])
    nan = torch.isnan(prob)
    with np.errstate(invalid="ignore"):
        ref = OL.forward(L2, idx, 0.1, off)
        rl = OL.backward(L2, host(clean[3]), off)
    assert np.array_equal(host(nan), np.isnan(ref[2])) and np.isnan(ref[0])
    assert bool(nan[s].all()) if bad != "inf" else bool(nan[s].any())
    assert torch.equal(prob[~nan.any(1)], clean[2][~nan.any(1)]) and int(nan.any(1).sum()) == 1
    assert np.isnan(rl[t]).all()
    other = torch.arange(T, device=dev) != t
    for plain, spoilt in grads:
        assert torch.isnan(spoilt[t]).all() and torch.equal(spoilt[other], plain[other])
