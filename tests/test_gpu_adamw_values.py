"""AdamW where a launch touches more than the package's 256 MB cache (other loads
there): bit for bit what small launches of the same elements, whose values the
oracle pins, give; the first and last elements also against the oracle itself."""
import numpy as np
import pytest
import torch

import moe_expert_routing_sqrt_amd as M
from oracle import adamw as OA

from gpu_util import host, need_gpu

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
H = dict(lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
CUT = 1 << 21                                    # elements of a small launch: a whole number of tiles


@pytest.mark.parametrize("p,g,bits,master", [("bf16", "f32", 32, True), ("bf16", "bf16", 8, True),
                                             ("f32", "f32", 32, False), ("f32", "bf16", 8, False),
                                             ("bf16", "bf16", 32, False), ("bf16", "f32", 8, True)])
def test_past_the_cache(p, g, bits, master):
    dev = need_gpu()
    n = 20_000_003 if bits == 32 else 34_000_003
    print(f"adamw of {n} {p} {g} bits={bits} master={master}", flush=True)
    each = (16 if bits == 32 else 4) + (4 if g == "f32" else 2) + (4 if p == "bf16" else 8) + (6 if master else 0)
    assert n * each > 256 * 2 ** 20
    gen = torch.Generator(device=dev).manual_seed(n)
    w = 0.05 * torch.randn(n, generator=gen, device=dev)
    param = w.to(DT[p])
    state = dict(master=[w.clone()] if master else None)
    if bits == 8:
        tiles = -(-n // 128)
        for name in ("m", "v"):
            c = torch.randint(0, 0x7F, (n,), generator=gen, device=dev, dtype=torch.uint8)
            if name == "m":
                c += 128 * torch.randint(0, 2, (n,), generator=gen, device=dev, dtype=torch.uint8)
            state[name] = [c]
            state[name + "_scale"] = [torch.exp2(torch.randint(-20, -10, (tiles,), generator=gen, device=dev).float())]
    else:
        state["m"] = [1e-3 * torch.randn(n, generator=gen, device=dev)]
        state["v"] = [1e-6 * torch.rand(n, generator=gen, device=dev)]
    grad = (1e-3 * torch.randn(n, generator=gen, device=dev)).to(DT[g])
    scale = torch.full((1,), 0.37, device=dev)
    small = {k: None if v is None else v[0].clone() for k, v in state.items()}
    sp = param.clone()
    first = {k: None if v is None else host(v[:CUT]) for k, v in small.items()}
    last = {k: None if v is None else host(v[-5000:]) for k, v in small.items()}
    p_first, p_last = host(sp[:CUT]), host(sp[-5000:])

    M.AdamW([param], [grad], step_count=6, **state, **H).step(scale)
    for at in range(0, n, CUT):                  # each under the cache's size
        e = slice(at, min(n, at + CUT))
        t = slice(at // 128, -(-e.stop // 128))
        pick = {k: None if v is None else [v[t if k.endswith("scale") else e]] for k, v in small.items()}
        M.AdamW([sp[e]], [grad[e]], step_count=6, **pick, **H).step(scale)
    torch.cuda.synchronize()
    assert torch.equal(param.view(torch.int32 if p == "f32" else torch.int16),
                       sp.view(torch.int32 if p == "f32" else torch.int16))
    for k, v in small.items():
        if v is not None:
            assert torch.equal(state[k][0], v), k
    if bits == 8:
        return                                   # a tile's scale needs whole tiles; test_gpu_adamw.py pins them
    for part, old, p0 in ((slice(0, CUT), first, p_first), (slice(n - 5000, n), last, p_last)):
        w0 = p0 if old["master"] is None else old["master"]
        rw, rm, rv, _ = OA.step(w0, host(grad[part]), old["m"], old["v"], lr=H["lr"], b1=0.9, b2=0.99, eps=1e-8, wd=0.1,
                                t=7, scale=0.37)
        got = host((state["master"][0] if master else param)[part])
        want = rw if master or p == "f32" else torch.from_numpy(np.ascontiguousarray(rw)).to(torch.bfloat16).float().numpy()
        assert np.array_equal(got, want) and np.array_equal(host(state["m"][0][part]), rm)
        assert np.array_equal(host(state["v"][0][part]), rv)
