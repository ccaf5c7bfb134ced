"""Temperatures at which a difference of logits beyond fp32 would still count are refused:
(x - max) / temperature is formed from the difference, which fp32 holds up to 3.4e38, and
below a temperature of 1e36 one larger than that is a probability of 0 (exp(-340)) in any
case.  No GPU: refused before any launch."""
import ctypes

import pytest

from moe_expert_routing_sqrt_amd import _lib

L = _lib.load()
INV = _lib.MOE_ERR_INVALID_ARG
X, I, TE, LO, RO, ST, LP, DX = (0x10000000 + (i << 20) for i in range(8))


@pytest.mark.parametrize("tau", [1.01e36, 1e37, 3e38])
def test_refused(tau):
    h = ctypes.byref(_lib.MoePolicyParams(tau, 0.2, 0.2, 0.0))
    assert L.moe_distill_loss(4, 8, 2, X, 0, I, TE, 0, tau, None, None, LO, RO, ST, None, 0, None) == INV
    assert L.moe_distill_loss_backward(4, 8, 2, X, 0, ST, I, TE, 0, tau, None, None, DX, 0, None) == INV
    assert L.moe_policy_loss(4, 8, X, 0, I, TE, TE, None, h, None, None, LO, RO, LP, ST, None, 0, None) == INV
    assert L.moe_policy_loss_backward(4, 8, X, 0, ST, I, TE, TE, None, h, None, None, DX, 0, None) == INV
    assert L.moe_token_logp(4, 8, X, 0, I, tau, LP, ST, None) == INV


@pytest.mark.parametrize("tau", [1e36, 1e35, 1.0, 1e-37])
def test_taken(tau):
    """(no rows: nothing is launched)"""
    assert L.moe_token_logp(0, 8, None, 0, None, tau, None, None, None) == 0
