"""A training step of one MoE block on synthetic data, timed by its parts.

    python -m moe_expert_routing_sqrt_amd.train_step [--workload flash] [--steps 10] [--states e4m3]
                                                     [--loss square|distill|policy] [--vocab 32768]

Each step: norm with the residual add, route, dispatch, experts, combine and
the balance loss; their backward for a squared error against a fixed target;
the auxiliary-loss-free bias update; AdamW on every weight.  With --loss distill
or policy the block is trained on token ids instead: embedding, block, norm and
tied head, and the distillation loss from a teacher's top logits or the policy loss
on the logits.  Prints the losses of the first and last step and the device time of
the parts.
"""
from __future__ import annotations

import argparse

import torch

from . import MoEBlock, MoELayer, TokenModel, distill_loss, policy_loss, token_logp


def make_block(cfg, dev, states: str, seed: int = 0, lr: float = 1e-3) -> MoEBlock:
    """A block of the given layer shape with random weights (bf16, fp32 router)."""
    g = torch.Generator(device=dev).manual_seed(seed)
    w = lambda *s: (0.02 * torch.randn(*s, generator=g, device=dev)).to(torch.bfloat16)  # noqa: E731
    d, f = cfg.d, cfg.d_ff
    layer = MoELayer(cfg.T, d, cfg.E, cfg.G, cfg.M, cfg.k, f, "bf16",
                     0.02 * torch.randn(d, cfg.E, generator=g, device=dev), torch.zeros(cfg.E, device=dev),
                     w(cfg.E, 2 * f, d), w(cfg.E, d, f), w(1, 2 * f, d), w(1, d, f), group_topk=cfg.gk)
    return MoEBlock(layer, torch.ones(d, device=dev), torch.zeros(d, device=dev), lr=lr, states=states)


def make_model(blk: MoEBlock, vocab: int, seed: int = 2) -> TokenModel:
    """The block between a table of `vocab` rows and itself as the head."""
    T, d, dev = blk.layer.T, blk.layer.d, blk.layer.bias.device
    g = torch.Generator(device=dev).manual_seed(seed)
    w = lambda *s: (0.02 * torch.randn(*s, generator=g, device=dev)).to(torch.bfloat16)  # noqa: E731
    return TokenModel(blk, w(vocab, d), w(T, d), torch.ones(d, device=dev), torch.zeros(d, device=dev))


class Tokens:
    """A fixed synthetic batch on token ids, and its loss."""

    def __init__(self, model: TokenModel, kind: str, seqs: torch.Tensor, top: int = 32, seed: int = 3):
        T, V, dev = model.block.layer.T, model.table.shape[0], model.table.device
        g = torch.Generator(device=dev).manual_seed(seed)
        draw = lambda *s: torch.randint(0, V, s, generator=g, device=dev, dtype=torch.int32)  # noqa: E731
        self.model, self.kind, self.seqs = model, kind, seqs
        self.ids, self.pos = draw(T), torch.arange(T, device=dev, dtype=torch.int32)
        self.out = {n: torch.empty(k, device=dev) for n, k in (("loss", 1), ("row_loss", T), ("stats", 2 * T))}
        self.top, self.teacher = draw(T, top), 2 * torch.randn(T, top, generator=g, device=dev)
        self.tokens, self.advantage = draw(T), torch.randn(T, generator=g, device=dev)
        self.logp, self.old = torch.empty(T, device=dev), None

    def forward(self):
        return self.model.forward(self.ids, self.pos, self.seqs)

    def loss(self, logits: torch.Tensor, factor: torch.Tensor) -> torch.Tensor:
        """The loss [1]; its gradient times factor is left over the logits."""
        if self.kind == "distill":
            return distill_loss(logits, self.top, self.teacher, 2.0, grad_loss=factor, dlogits=logits, **self.out)[0]
        if self.old is None:  # the first step's policy is the one that sampled
            self.old = token_logp(logits, self.tokens)[0]
        return policy_loss(logits, self.tokens, self.old, self.advantage, self.old, kl=0.05, grad_loss=factor,
                           dlogits=logits, logp=self.logp, **self.out)[0]


def main(argv=None) -> dict:
    from moe_inputs import configs

    ap = argparse.ArgumentParser()
    ap.add_argument("--workload", default="flash", help="a bf16 shape of moe_inputs.configs")
    ap.add_argument("--tokens", type=int, default=None, help="instead of the workload's")
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--states", choices=("f32", "e4m3"), default="e4m3")
    ap.add_argument("--lr", type=float, default=None, help="1e-3; with --loss policy 1e-5, which keeps to its clip")
    ap.add_argument("--loss", choices=("square", "distill", "policy"), default="square")
    ap.add_argument("--vocab", type=int, default=32768, help="with --loss distill or policy")
    a = ap.parse_args(argv)
    lr = a.lr if a.lr is not None else 1e-5 if a.loss == "policy" else 1e-3
    cfg = configs.get(a.workload)
    if a.tokens is not None:
        cfg = cfg.with_(T=a.tokens)
    dev = torch.device("cuda")
    blk = make_block(cfg, dev, a.states, lr=lr)
    g = torch.Generator(device=dev).manual_seed(1)
    new = lambda: torch.randn(cfg.T, cfg.d, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    delta, stream, target = new(), new(), new()
    seqs = torch.arange(a.sequences + 1, device=dev, dtype=torch.int32) * cfg.T // a.sequences
    seqs = seqs.to(torch.int32)
    # d_out is the gradient of T times the loss; the balance loss's carries T too
    factor = torch.full((1,), float(cfg.T), device=dev)
    scale = 1.0 / factor
    data = None
    if a.loss != "square":
        model = make_model(blk, a.vocab)
        data = Tokens(model, a.loss, seqs)
    names = ("forward", "loss", "backward", "bias update", "optimizer")
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(len(names) + 1)]
    times = dict.fromkeys(names, 0.0)
    errs = []
    for i in range(a.steps):
        ev[0].record()
        if data is None:
            out, _ = blk.forward(delta, stream, seqs)
            ev[1].record()
            diff = out - target
            err = diff.float().square().mean()
            ev[2].record()
            blk.backward(diff, grad_loss=factor)
        else:
            logits = data.forward()
            ev[1].record()
            err = data.loss(logits, factor)
            ev[2].record()
            model.backward(logits, grad_loss=factor)
        ev[3].record()
        blk.layer.update_bias(1e-3)
        ev[4].record()
        (blk if data is None else model).step(scale)
        ev[5].record()
        torch.cuda.synchronize()
        errs.append((float(err), float(blk.loss)))
        if i >= min(2, a.steps - 1):  # the first steps make the buffers
            for j, n in enumerate(names):
                times[n] += ev[j].elapsed_time(ev[j + 1])
    timed = max(1, a.steps - min(2, a.steps - 1))
    ms = {n: t / timed for n, t in times.items()}
    print(f"{cfg.name}: T={cfg.T} d={cfg.d} E={cfg.E} d_ff={cfg.d_ff}, states {a.states}")
    what = {"square": "squared error", "distill": "distillation loss", "policy": "policy loss"}[a.loss]
    if data is not None:
        print(f"on token ids: vocabulary of {a.vocab}")
    print(f"{what} {errs[0][0]:.4f} -> {errs[-1][0]:.4f}, balance loss {errs[0][1]:.3e} -> {errs[-1][1]:.3e}")
    print("ms a step: " + ", ".join(f"{n} {t:.3f}" for n, t in ms.items()))
    return {"errors": errs, "ms": ms}


if __name__ == "__main__":
    main()
