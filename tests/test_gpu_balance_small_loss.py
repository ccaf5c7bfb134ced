"""A balance loss far below 1 keeps fp32's relative precision: few of many
sequences hold tokens, or the selected experts are improbable.

Tolerance, u = 2^-24: a probability is within 28u, a mean of up to 64 tokens adds
a chain of at most 24 and a product 1u, f 3u, and the sum over experts and
work-groups at most 64 additions: 128u of a sum of positive terms."""
import numpy as np
import pytest
import torch

import moe_expert_routing_sqrt_amd as M
from oracle import balance_loss as OL

from gpu_util import dev_f32, dev_i32, host, need_gpu

pytestmark = pytest.mark.gpu

REL = 128 * 2.0 ** -24


@pytest.mark.parametrize("n", [300, 1024, 4096, 16384, 65535])
@pytest.mark.parametrize("E", [100, 256])
def test_one_sequence_among_empty_ones(n, E):
    dev = need_gpu()
    print(f"one of {n} sequences, E={E}", flush=True)
    T, k = 50, 4
    for seed in range(4):
        rng = np.random.default_rng(seed)
        L = rng.normal(size=(T, E)).astype(np.float32)
        idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
        at = int(rng.integers(0, n))
        off = np.where(np.arange(n + 1) <= at, 0, T).astype(np.int32)
        alone = OL.forward(L, idx, 1.0)
        loss, counts, prob, dprob = M.balance_loss(M.shape(T, 1, E, 1, 1, k, 1, 1), dev_f32(L, dev),
                                                   dev_i32(idx, dev), 1.0, seq_offsets=dev_i32(off, dev))
        torch.cuda.synchronize()
        assert np.array_equal(host(counts[at]), alone[1][0]) and int(counts.sum()) == T * k
        assert np.abs(host(prob[at]) / alone[2][0] - 1).max() <= REL
        assert abs(float(loss) * n / alone[0] - 1) <= REL, (seed, float(loss) * n / alone[0] - 1)


@pytest.mark.parametrize("T,E,n", [(50, 64, 2), (500, 64, 1), (500, 64, 5), (500, 256, 40), (200, 600, 3), (130, 20, 1)])
@pytest.mark.parametrize("low", [-10.0, -40.0, -100.0])
def test_improbable_selections(T, E, n, low):
    dev = need_gpu()
    print(f"selections at logit {low}: T={T} E={E} n={n}", flush=True)
    rng = np.random.default_rng(T + E)
    L = rng.normal(size=(T, E)).astype(np.float32)
    L[:, :2] += low
    idx = np.tile(np.array([0, 1], dtype=np.int32), (T, 1))
    off = (np.arange(n + 1) * T // n).astype(np.int32)
    ref = OL.forward(L, idx, 1.0, off)
    loss = M.balance_loss(M.shape(T, 1, E, 1, 1, 2, 1, 1), dev_f32(L, dev), dev_i32(idx, dev), 1.0,
                          seq_offsets=dev_i32(off, dev))[0]
    # a mean of T / n tokens: chains of 4 in a wave, 16 waves, then T / 64 tiles
    rel = REL + (T / n / 64) * 2.0 ** -24
    assert abs(float(loss) / ref[0] - 1) <= rel, float(loss) / ref[0] - 1


def test_shares_of_every_size_together():
    """Sequences whose losses lie far apart: the same bits on every call, with other
    work in between."""
    dev = need_gpu()
    T, E, k, n = 3000, 256, 2, 30
    rng = np.random.default_rng(3)
    L = rng.normal(size=(T, E)).astype(np.float32)
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    L[::3, 32:] -= 30.0                       # the experts of most slices improbable in some tokens,
    L[1500:, 64:] -= 60.0                     # and in all of half of the sequences
    off = (np.arange(n + 1) * T // n).astype(np.int32)
    ref = OL.forward(L, idx, 1.0, off)
    args = (M.shape(T, 1, E, 1, 1, k, 1, 1), dev_f32(L, dev), dev_i32(idx, dev), 1.0)
    first = M.balance_loss(*args, seq_offsets=dev_i32(off, dev))
    assert abs(float(first[0]) / ref[0] - 1) <= REL
    for i in range(20):
        torch.randn(1 << (10 + i % 8), device=dev).sum()
        again = M.balance_loss(*args, seq_offsets=dev_i32(off, dev))
        assert all(torch.equal(p, q) for p, q in zip(first, again)), i
