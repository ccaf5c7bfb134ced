"""The balance loss's largest number of tokens (no GPU: the host checks alone)."""
import ctypes

from moe_expert_routing_sqrt_amd import _lib

L = _lib.load()
FAKE = 0x1000


def test_most_tokens_of_a_launch():
    """The gradient takes 256 threads for 4 tokens (E > 128), and a launch takes
    fewer than 2^32 threads: 4 (2^24 - 1) tokens at most."""
    most = 4 * (2 ** 24 - 1)
    ok, over = _lib.MoeShape(most, 1, 256, 1, 1, 4, 1, 1), _lib.MoeShape(most + 1, 1, 256, 1, 1, 4, 1, 1)
    assert L.moe_balance_loss_workspace_size(ctypes.byref(ok), 1) > 0
    assert L.moe_balance_loss_workspace_size(ctypes.byref(over), 1) == 0
    for T in (most + 1, most + 2, most + 3, 2 ** 26):
        sh = _lib.MoeShape(T, 1, 256, 1, 1, 4, 1, 1)
        assert L.moe_balance_loss_backward(ctypes.byref(sh), FAKE, None, None, 1, None, FAKE, None, None, FAKE,
                                           None) == _lib.MOE_ERR_UNSUPPORTED
