"""A training step of one MoE block on synthetic data, timed by its parts.

    python -m moe_expert_routing_sqrt_amd.train_step [--workload flash] [--steps 10] [--states e4m3]

Each step: norm with the residual add, route, dispatch, experts, combine and
the balance loss; their backward for a squared error against a fixed target;
the auxiliary-loss-free bias update; AdamW on every weight.  Prints the losses
of the first and last step and the device time of the parts.
"""
from __future__ import annotations

import argparse

import torch

from . import MoEBlock, MoELayer


def make_block(cfg, dev, states: str, seed: int = 0, lr: float = 1e-3) -> MoEBlock:
    """A block of the given layer shape with random weights (bf16, fp32 router)."""
    g = torch.Generator(device=dev).manual_seed(seed)
    w = lambda *s: (0.02 * torch.randn(*s, generator=g, device=dev)).to(torch.bfloat16)  # noqa: E731
    d, f = cfg.d, cfg.d_ff
    layer = MoELayer(cfg.T, d, cfg.E, cfg.G, cfg.M, cfg.k, f, "bf16",
                     0.02 * torch.randn(d, cfg.E, generator=g, device=dev), torch.zeros(cfg.E, device=dev),
                     w(cfg.E, 2 * f, d), w(cfg.E, d, f), w(1, 2 * f, d), w(1, d, f), group_topk=cfg.gk)
    return MoEBlock(layer, torch.ones(d, device=dev), torch.zeros(d, device=dev), lr=lr, states=states)


def main(argv=None) -> dict:
    from moe_inputs import configs

    ap = argparse.ArgumentParser()
    ap.add_argument("--workload", default="flash", help="a bf16 shape of moe_inputs.configs")
    ap.add_argument("--tokens", type=int, default=None, help="instead of the workload's")
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--states", choices=("f32", "e4m3"), default="e4m3")
    ap.add_argument("--lr", type=float, default=1e-3)
    a = ap.parse_args(argv)
    cfg = configs.get(a.workload)
    if a.tokens is not None:
        cfg = cfg.with_(T=a.tokens)
    dev = torch.device("cuda")
    blk = make_block(cfg, dev, a.states, lr=a.lr)
    g = torch.Generator(device=dev).manual_seed(1)
    new = lambda: torch.randn(cfg.T, cfg.d, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    delta, stream, target = new(), new(), new()
    seqs = torch.arange(a.sequences + 1, device=dev, dtype=torch.int32) * cfg.T // a.sequences
    seqs = seqs.to(torch.int32)
    # d_out is the gradient of T times the loss; the balance loss's carries T too
    factor = torch.full((1,), float(cfg.T), device=dev)
    scale = 1.0 / factor
    names = ("forward", "loss", "backward", "bias update", "optimizer")
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(len(names) + 1)]
    times = dict.fromkeys(names, 0.0)
    errs = []
    for i in range(a.steps):
        ev[0].record()
        out, _ = blk.forward(delta, stream, seqs)
        ev[1].record()
        diff = out - target
        err = diff.float().square().mean()
        ev[2].record()
        blk.backward(diff, grad_loss=factor)
        ev[3].record()
        blk.layer.update_bias(1e-3)
        ev[4].record()
        blk.step(scale)
        ev[5].record()
        torch.cuda.synchronize()
        errs.append((float(err), float(blk.loss)))
        if i >= min(2, a.steps - 1):  # the first steps make the buffers
            for j, n in enumerate(names):
                times[n] += ev[j].elapsed_time(ev[j + 1])
    timed = max(1, a.steps - min(2, a.steps - 1))
    ms = {n: t / timed for n, t in times.items()}
    print(f"{cfg.name}: T={cfg.T} d={cfg.d} E={cfg.E} d_ff={cfg.d_ff}, states {a.states}")
    print(f"squared error {errs[0][0]:.4f} -> {errs[-1][0]:.4f}, balance loss {errs[0][1]:.3e} -> {errs[-1][1]:.3e}")
    print("ms a step: " + ", ".join(f"{n} {t:.3f}" for n, t in ms.items()))
    return {"errors": errs, "ms": ms}


if __name__ == "__main__":
    main()
