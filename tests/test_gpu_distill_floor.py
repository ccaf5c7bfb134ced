"""GPU: how small a distillation loss may be before its error hides it.

A row's loss is sum p (log p - log q), whose logarithms are those of two fp32 sums of
exponentials: it carries their relative errors as an absolute one, however small it is.
With U = 2^-24, V = K = 32 (one wave, 4 logits a lane) and z = (x - max) of student or
teacher:
  an exponential  U (2 |z| + 2): the difference's and the exponent's rounding, its own
  its sum         U (2 mean |z| + 2) and 3 + 6 additions
  a logarithm     U of its own and U where the exponent's share is added
  a probability   U (2 |zt| + 2), its sum's and a division's, times the row's |log p - log q|
Together with the product's and the store's rounding that is the tolerance here, about
2e-6; at gaps of 0.1 and 0.01 it is a part of the loss, so that neither 0 nor twice the
loss passes.  Below, only the absolute error is held."""
import numpy as np
import pytest
import torch

import moe_expert_routing_sqrt_amd as M
from oracle import vocab_loss as OV

from gpu_util import host, need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _spread(x):
    z = x - x.max(1, keepdims=True)
    e = np.exp(z)
    return (e * -z).sum(1) / e.sum(1)


@pytest.mark.parametrize("gap", [1e-1, 1e-2, 1e-3, 1e-5, 0.0])
@pytest.mark.parametrize("tau", [1.0, 2.0])
def test_small_losses(gap, tau):
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(8)
    n = 512
    x = torch.randn(n, 32, generator=g, device=dev) * tau
    idx = torch.arange(32, device=dev, dtype=torch.int32).repeat(n, 1)
    t = x + gap * tau * torch.randn(n, 32, generator=g, device=dev)
    _, row, _, dx = M.distill_loss(x, idx, t, tau, torch.ones(n, device=dev), with_grad=True)
    h, th = host(x).astype(np.float64), host(t).astype(np.float64)
    ref = OV.distill(h, host(idx), th, tau, np.ones(n))
    zs, zt = _spread(h / tau), _spread(th / tau)
    logs = np.abs((th - h) / tau) + np.abs(np.log(np.exp(h / tau).sum(1) / np.exp(th / tau).sum(1)))[:, None]
    p = np.exp(th / tau) / np.exp(th / tau).sum(1, keepdims=True)
    z = (th.max(1, keepdims=True) - th) / tau
    own = (p * logs * (2 * z + 2 + (2 * zt + 12)[:, None])).sum(1)
    tol = U * tau ** 2 * (2 * zs + 2 * zt + 2 * 11 + 4 + own) + 2 * U * np.abs(ref["row_loss"])
    err = host(row).astype(np.float64) - ref["row_loss"]
    print(f"gap {gap} tau {tau}: loss {ref['row_loss'].mean():.2e}, error rms {np.sqrt((err ** 2).mean()):.1e}, "
          f"largest {np.abs(err).max():.1e}, tolerance {tol.max():.1e}", flush=True)
    assert (np.abs(err) <= tol).all()
    if gap >= 1e-2:
        assert (ref["row_loss"] > tol).all()
    # the gradient tau (q - p): each probability's relative error
    q = np.exp(h / tau) / np.exp(h / tau).sum(1, keepdims=True)
    zq = (h.max(1, keepdims=True) - h) / tau
    allowed = U * tau * (q * (2 * zq + 16 + 2 * zs[:, None]) + p * (2 * z + 16 + 2 * zt[:, None]))
    assert (np.abs(host(dx) - ref["dlogits"]) <= allowed).all()
