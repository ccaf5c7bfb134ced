"""The balance loss's gradient at the largest number of tokens it takes."""
import pytest
import torch

import moe_expert_routing_sqrt_amd as M

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def test_most_tokens():
    """2^26 - 4 tokens of 129 experts (a wave each): around both ends as the same
    tokens alone."""
    dev = need_gpu()
    if torch.cuda.mem_get_info()[0] < 90 * 2 ** 30:
        pytest.skip("needs 90 GB of GPU memory")
    T, E, part = 2 ** 26 - 4, 129, 1000
    logits = torch.zeros(T, E, device=dev)
    for rows in (slice(0, part), slice(T - part, T)):
        logits[rows] = 2 * torch.randn(part, E, device=dev)
    dprob = torch.rand(1, E, device=dev)
    dl = M.balance_loss_backward(M.shape(T, 1, E, 1, 1, 1, 1, 1), logits, dprob)
    small = M.shape(part, 1, E, 1, 1, 1, 1, 1)
    for rows in (slice(0, part), slice(T - part, T)):
        assert torch.equal(dl[rows], M.balance_loss_backward(small, logits[rows].contiguous(), dprob))
    zero = M.balance_loss_backward(M.shape(1, 1, E, 1, 1, 1, 1, 1), torch.zeros(1, E, device=dev), dprob)
    for at in range(part, T - part, 1 << 22):
        rows = dl[at:min(at + (1 << 22), T - part)]
        assert bool((rows == zero).all()), at
