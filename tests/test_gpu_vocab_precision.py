"""GPU: what the softmax's exponent holds of log2(e)/tau."""
import math

import numpy as np
import pytest
import torch

import moe_expert_routing_sqrt_amd as M

from gpu_util import host, need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
# log2(e)/tau in the middle between two fp32 numbers, where rounding it takes 2^-24 of it away or adds it
TAUS = [math.log2(math.e) / (1 + k * U) for k in (1, 3)]


@pytest.mark.parametrize("tau", TAUS)
@pytest.mark.parametrize("T,V", [(64, 20000), (16, 140003)])
def test_sums_have_no_common_error(tau, T, V):
    """One logit at 0 and all others about 11 tau below it, most of the sum.  With the
    exponent's factor rounded to fp32 every term is off by 2^-24 of some 10 in the same
    direction, 3e-7 of the sum and more.  With its low part the exponent is the fp32 number
    nearest to x log2(e)/tau (but for 2^-48 of it), which is what the sums are held to: that
    last rounding is at most 2^-21 of an exponent of 8 to 16 and need not have either sign
    alike (the factor here is 1 + k 2^-24, so that it moves an x of 24 bits by 0.5 to 3 units
    in its last place, whose fractions are not evenly spread: 1.7e-7 of a sum at k = 3).
    What is left and may have one sign is the exponential's own error, at most 2 U; the
    additions' rounding has either sign over thousands of terms."""
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(V)
    low = -12.0 if V > 100000 else -10.5
    x = torch.empty(T, V, device=dev).uniform_(low * tau, (low + 2) * tau, generator=g)
    x[:, 5] = 0
    idx = torch.full((T, 1), 7, dtype=torch.int32, device=dev)
    stats = M.distill_loss(x, idx, torch.zeros(T, 1, device=dev), tau)[2]
    exponent = (host(x).astype(np.float64) * (math.log2(math.e) / tau)).astype(np.float32)
    want = np.exp2(exponent.astype(np.float64)).sum(1)
    rel = host(stats)[:, 1] / want - 1
    print("mean relative error of the sums", rel.mean(), flush=True)
    assert (host(stats)[:, 0] == 0).all() and abs(rel.mean()) <= 2 * U + U / 4
