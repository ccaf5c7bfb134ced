"""The two ends of a training step on tokens, as a benchmark: the embedding
lookup and its gradient, and the losses on a vocabulary's logits with their
gradients: distillation from a teacher's top logits, and the clipped policy
loss with a KL term.

`run` computes them in plain torch (fp32, rounded once at the end; the few
numbers a row of the policy loss has in fp64, as its derivative jumps at the
clip's border), or through this package's entry points where `own` is true.
`exact` evaluates the same definitions in fp64, the losses' gradients by
automatic differentiation.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
ZIPF = 2.7          # token v of a vocabulary has about 1 / (v + ZIPF) of the text
CLIP = (0.2, 0.28)  # the ratio's lower and upper clip
MASKED = 0.1        # share of tokens that carry no loss, where a case weights its tokens


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decoding batch's rows of the table: eight tokens, latency is all
        dict(name="embed_decode", op="embed_fwd", T=8, V=131072, d=7168, x="bf16", y="bf16", pad=False),
        # a packed batch with padding ids, fp32 table to bf16 rows
        dict(name="embed_f32", op="embed_fwd", T=4096, V=32768, d=2048, x="f32", y="bf16", pad=True),
        # the 256-expert layer's batch, four sequences of 4096
        dict(name="embed_large", op="embed_fwd", T=16384, V=131072, d=7168, x="bf16", y="bf16", pad=False),
        # an odd batch, vocabulary and width with padding ids: nothing is aligned
        dict(name="embed_bwd_odd", op="embed_bwd", T=1000, V=5003, d=1001, x="f32", y="f32", pad=True, add=False),
        # a tied table: the head's gradient is there, the touched rows are added to
        dict(name="embed_bwd_tied", op="embed_bwd", T=16384, V=65536, d=2048, x="bf16", y="f32", pad=False, add=True),
        # the whole gradient of the 256-expert layer's table, untouched rows zero
        dict(name="embed_bwd_large", op="embed_bwd", T=16384, V=131072, d=7168, x="bf16", y="f32", pad=False,
             add=False),
        # a short answer's tokens, loss and gradient in one call
        dict(name="distill_small", op="distill", T=64, V=32000, K=32, x="bf16", y="bf16", tau=1.0, weight=True,
             ragged=False),
        # a batch over a large vocabulary, loss and gradient in one call
        dict(name="distill_large", op="distill", T=4096, V=131072, K=64, x="bf16", y="bf16", tau=2.0, weight=False,
             ragged=False),
        # the gradient by itself, an odd vocabulary in fp32, rows with few or no teacher entries
        dict(name="distill_bwd_odd", op="distill_bwd", T=1500, V=50001, K=20, x="f32", y="f32", tau=1.5, weight=True,
             ragged=True),
        # scoring a decoding batch: the loss alone
        dict(name="policy_fwd_small", op="policy_fwd", T=32, V=65536, x="bf16", y="bf16", tau=1.0, weight=True,
             kl=0.0),
        # a policy update's batch, loss and gradient in one call
        dict(name="policy_large", op="policy", T=8192, V=65536, x="bf16", y="bf16", tau=1.0, weight=True, kl=0.05),
        # the gradient by itself: fp32 logits, bf16 gradient for the head's product, odd vocabulary
        dict(name="policy_bwd_odd", op="policy_bwd", T=2048, V=100003, x="f32", y="bf16", tau=0.7, weight=True,
             kl=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "distill", "distill_fwd", "distill_bwd", "policy", "policy_fwd",
                     "policy_bwd"])
    x, y = rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"])
    if op.startswith("embed"):
        d = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            d = max(64, d // 64 * 64)
        V = _log(rng, 500, max(501, min(131072, 131072 * 3584 // d)))
        c = dict(op=op, T=_log(rng, 1, min(32768, 16384 * 7168 // 2 // d)), V=V, d=d, x=x, y=y,
                 pad=rng.random() < 0.5)
        if op == "embed_bwd":
            c["add"] = rng.random() < 0.5
        return c
    V = _log(rng, 200, 131072)
    if rng.random() < 0.5:
        V = max(256, V // 256 * 256)
    c = dict(op=op, T=_log(rng, 1, max(1, min(16384, (1 << 28) // V))), V=V, x=x, y=y,
             tau=rng.choice([1.0, 1.0, 0.7, 2.0, 4.0]), weight=rng.random() < 0.6)
    if op.startswith("distill"):
        c.update(K=min(V, rng.randint(1, 128)), ragged=rng.random() < 0.4)
    else:
        c["kl"] = rng.choice([0.0, 0.02, 0.1])
    return c


def _distinct(case):
    """How many rows of the table a batch touches, on average."""
    v = np.arange(case["V"], dtype=np.float64) + ZIPF
    p = np.log((v + 1) / v) / math.log((case["V"] + ZIPF) / ZIPF)
    return float((1 - (1 - p) ** case["T"]).sum())


def work(case):
    op, T, V, x, y = case["op"], case["T"], case["V"], BYTES[case["x"]], BYTES[case["y"]]
    if op == "embed_fwd":
        d = case["d"]
        return {"bytes": 4 * T + d * (x * _distinct(case) + y * T), "flops": T * d}
    if op == "embed_bwd":
        d = case["d"]
        rows = 2 * _distinct(case) if case["add"] else V
        return {"bytes": 4 * T + d * (x * T + y * rows), "flops": 2 * T * d}
    kept = (1 - MASKED) * T if case["weight"] else T
    grad = not op.endswith("fwd")
    few = T * (8 * case["K"] + 16) if op.startswith("distill") else 40 * T
    return {"bytes": V * (x * kept + (y * T if grad else 0)) + few, "flops": V * kept * (7 if grad else 4)}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _tokens(g, n, V):
    """Token ids as text has them: few common, many rare, in no order."""
    u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
    rank = (ZIPF * ((V + ZIPF) / ZIPF) ** u - ZIPF).long().clamp(0, V - 1)
    return torch.randperm(V, generator=g, device=DEV)[rank].to(torch.int32)


def _prepare_embed(case, g):
    T, V, d = case["T"], case["V"], case["d"]
    ids = _tokens(g, T, V)
    if case["pad"]:
        ids[torch.rand(T, generator=g, device=DEV) < 0.15] = -1
    st = dict(case=case, ids=ids, scale=math.sqrt(d))
    if case["op"] == "embed_fwd":
        st["table"] = (torch.randn(V, d, generator=g, device=DEV) * 0.02).to(DT[case["x"]])
    else:
        st["dy"] = (torch.randn(T, d, generator=g, device=DEV) * 0.02).to(DT[case["x"]])
        if case["add"]:
            st["table"] = (torch.randn(V, d, generator=g, device=DEV) * 0.1).to(DT[case["y"]])
    return st


def _blocks(T, V):
    """Row blocks of about 64 M logits."""
    n = max(1, (1 << 26) // V)
    return [slice(a, min(T, a + n)) for a in range(0, T, n)]


def _prepare_loss(case, g):
    T, V, tau = case["T"], case["V"], case["tau"]
    # peaked rows: a broad spread and some likely tokens; the vocabulary's last columns are padding
    x = torch.empty(T, V, device=DEV, dtype=DT[case["x"]])
    some = torch.randn(V, generator=g, device=DEV)
    for r in _blocks(T, V):
        z = torch.randn(x[r].shape, generator=g, device=DEV)
        x[r] = (1.5 * z + some + 0.25 * z * z * z.abs()).to(x.dtype)
    x[:, V - V // 64:] = float("-inf")
    st = dict(case=case, x=x, grad=torch.full((1,), 0.5, device=DEV), weight=None)
    if case["weight"]:
        w = (torch.rand(T, generator=g, device=DEV) >= MASKED).float()
        st["weight"] = w / w.sum().clamp(min=1)
    if case["op"].startswith("distill"):
        K = case["K"]
        t = torch.empty(T, K, device=DEV)
        idx = torch.empty(T, K, device=DEV, dtype=torch.int32)
        for r in _blocks(T, V):
            z = x[r].float() + torch.randn(x[r].shape, generator=g, device=DEV)
            t[r], i = z.topk(K, dim=1)
            idx[r] = i.to(torch.int32)
        if case["ragged"]:  # rows of 0 to K entries
            keep = torch.randint(0, K + 1, (T, 1), generator=g, device=DEV)
            idx[torch.arange(K, device=DEV) >= keep] = -1
        st.update(idx=idx, t=t)
    else:
        tok = torch.empty(T, device=DEV, dtype=torch.int32)
        logp = torch.empty(T, device=DEV, dtype=torch.float64)
        for r in _blocks(T, V):
            z = x[r].double() / tau
            gum = -torch.log(-torch.log(torch.rand(z.shape, generator=g, device=DEV).clamp(1e-20, 1 - 1e-7)))
            i = (z + gum).argmax(1)
            tok[r] = i.to(torch.int32)
            logp[r] = z.gather(1, i[:, None])[:, 0] - torch.logsumexp(z, 1)
        move = 0.15 * torch.randn(T, generator=g, device=DEV, dtype=torch.float64)  # logp - old_logp
        for border in (math.log(1 - CLIP[0]), math.log(1 + CLIP[1])):  # where the derivative jumps
            move = torch.where((move - border).abs() < 1e-3, move + 4e-3, move)
        st.update(tok=tok, old=(logp - move).float(), adv=torch.randn(T, generator=g, device=DEV))
        st["ref"] = (logp + 0.2 * torch.randn(T, generator=g, device=DEV)).float() if case["kl"] else None
    if case["op"].endswith("bwd"):  # what the forward left: each row's maximum and its sum of exponentials
        st["stats"] = torch.empty(T, 2, device=DEV)
        for r in _blocks(T, V):
            z = x[r].double()
            m = z.amax(1, keepdim=True)
            st["stats"][r] = torch.stack([m[:, 0], torch.exp((z - m) / tau).sum(1)], 1).float()
    return st


def prepare(case, seed):
    g = _gen(seed)
    return _prepare_embed(case, g) if case["op"].startswith("embed") else _prepare_loss(case, g)


# ---------------------------------------------------------------- plain forms

def _plain_embed_fwd(st):
    ids = st["ids"].long()
    inside = ids >= 0
    out = st["table"][ids.clamp(min=0)].float() * st["scale"]
    return dict(out=torch.where(inside[:, None], out, 0.0).to(DT[st["case"]["y"]]))


def _plain_embed_bwd(st):
    c = st["case"]
    ids = st["ids"].long()
    total = torch.zeros(c["V"] + 1, c["d"], device=DEV)
    total.index_add_(0, torch.where(ids >= 0, ids, c["V"]), st["dy"].float())
    total = total[:-1] * st["scale"]
    if not c["add"]:
        return dict(d_table=total.to(DT[c["y"]]))
    st["table"].copy_(st["table"].float() + total)
    return dict(d_table=st["table"])


def _weight(st):
    T = st["case"]["T"]
    return torch.full((T,), 1.0 / T, device=DEV) if st["weight"] is None else st["weight"]


def _softmax(st, counted):
    """exp((x - max) / tau), and the rows' maxima and sums (0 where a row does not count)"""
    x = torch.where(counted[:, None], st["x"].float(), 0.0)
    m = x.amax(1, keepdim=True)
    e = torch.exp((x - m) / st["case"]["tau"])
    s = e.sum(1, keepdim=True)
    stats = torch.where(counted[:, None], torch.cat([m, s], 1), 0.0)
    return e, m, s, stats


def _plain_distill(st):
    c = st["case"]
    tau, op = c["tau"], c["op"]
    w = _weight(st)
    idx = st["idx"].long()
    ok = idx >= 0
    counted = (w != 0) & ok.any(1)
    idx = idx.clamp(min=0)
    ok = ok & counted[:, None]
    t = torch.where(ok, st["t"].float(), float("-inf"))
    u = torch.where(counted[:, None], t - t.amax(1, keepdim=True), float("-inf")) / tau
    ts = torch.exp(u).sum(1, keepdim=True)
    p = torch.where(ok, torch.exp(u) / ts, 0.0)
    if op == "distill_bwd":
        m, s = torch.where(counted[:, None], st["stats"], 1.0).split(1, 1)
        e = torch.exp((torch.where(counted[:, None], st["x"].float(), 0.0) - m) / tau)
    else:
        e, m, s, stats = _softmax(st, counted)
        zs = (torch.where(ok, st["x"].gather(1, idx).float(), 0.0) - m) / tau
        logs = u - torch.log(ts) - (zs - torch.log(s))
        row = torch.where(ok, p * logs, 0.0).sum(1) * tau ** 2
        out = dict(loss=(w * row).sum().reshape(1), row_loss=row, stats=stats)
        if op == "distill_fwd":
            return out
    k = torch.where(counted, st["grad"] * w * tau, 0.0)[:, None]
    dx = k * (e / s)
    dx.scatter_add_(1, idx, -k * p)
    dx = dx.to(DT[c["y"]])
    return dict(dlogits=dx) if op == "distill_bwd" else dict(dlogits=dx, **out)


def _plain_policy(st):
    c = st["case"]
    tau, op = c["tau"], c["op"]
    w = _weight(st)
    counted = w != 0
    if op == "policy_bwd":
        m, s = torch.where(counted[:, None], st["stats"], 1.0).split(1, 1)
        e = torch.exp((torch.where(counted[:, None], st["x"].float(), 0.0) - m) / tau)
    else:
        e, m, s, stats = _softmax(st, counted)
    at = st["tok"].long()[:, None]
    logp = (st["x"].gather(1, at).double() - m.double()) / tau - torch.log(s.double())
    logp = torch.where(counted, logp[:, 0], 0.0)
    r = torch.exp(logp - st["old"].double())
    adv = st["adv"].double()
    free, cut = r * adv, r.clamp(1 - CLIP[0], 1 + CLIP[1]) * adv
    row, slope = -torch.minimum(free, cut), torch.where(free <= cut, -free, 0.0)
    if c["kl"]:
        d = st["ref"].double() - logp
        row = row + c["kl"] * (torch.expm1(d) - d)
        slope = slope - c["kl"] * torch.expm1(d)
    row = torch.where(counted, row, 0.0)
    out = dict(loss=(w.double() * row).sum().float().reshape(1), row_loss=row.float(), logp=logp.float())
    if op == "policy_fwd":
        return dict(stats=stats, **out)
    k = torch.where(counted, st["grad"] * w * slope / tau, 0.0).float()[:, None]
    dx = -k * (e / s)
    dx.scatter_add_(1, at, k)
    dx = dx.to(DT[c["y"]])
    return dict(dlogits=dx) if op == "policy_bwd" else dict(dlogits=dx, stats=stats, **out)


# ---------------------------------------------------------------- the framework's operators

def _own_run(st):
    import moe_expert_routing_sqrt_amd as M
    c = st["case"]
    op, y = c["op"], DT[c["y"]]
    if op == "embed_fwd":
        return dict(out=M.embedding(st["ids"], st["table"], scale=st["scale"], out_dtype=y))
    if op == "embed_bwd":
        if c["add"]:
            return dict(d_table=M.embedding_backward(st["dy"], st["ids"], c["V"], scale=st["scale"],
                                                     d_table=st["table"], accumulate=True))
        return dict(d_table=M.embedding_backward(st["dy"], st["ids"], c["V"], scale=st["scale"], dtype=y))
    grad = dict(grad_loss=st["grad"], grad_dtype=y)
    if op == "distill_bwd":
        return dict(dlogits=M.distill_loss_backward(st["x"], st["stats"], st["idx"], st["t"], temperature=c["tau"],
                                                    weight=st["weight"], **grad))
    if op.startswith("distill"):
        more = {} if op == "distill_fwd" else dict(with_grad=True, **grad)
        loss, row, stats, dx = M.distill_loss(st["x"], st["idx"], st["t"], temperature=c["tau"], weight=st["weight"],
                                              **more)
        out = dict(loss=loss, row_loss=row, stats=stats)
    else:
        args = dict(ref_logp=st["ref"], clip=CLIP, kl=c["kl"], temperature=c["tau"], weight=st["weight"])
        if op == "policy_bwd":
            return dict(dlogits=M.policy_loss_backward(st["x"], st["stats"], st["tok"], st["old"], st["adv"], **args,
                                                       **grad))
        more = {} if op == "policy_fwd" else dict(with_grad=True, **grad)
        loss, row, logp, stats, dx = M.policy_loss(st["x"], st["tok"], st["old"], st["adv"], **args, **more)
        out = dict(loss=loss, row_loss=row, logp=logp, stats=stats)
    return out if dx is None else dict(dlogits=dx, **out)


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op.startswith("distill"):
        return _plain_distill(state)
    if op.startswith("policy"):
        return _plain_policy(state)
    return _plain_embed_fwd(state) if op == "embed_fwd" else _plain_embed_bwd(state)


# ---------------------------------------------------------------- 64 bits

def _exact_embed(st, c):
    ids = st["ids"].long()
    if c["op"] == "embed_fwd":
        out = torch.zeros(c["T"], c["d"], dtype=torch.float64, device=DEV)
        at = (ids >= 0).nonzero()[:, 0]
        out[at] = st["scale"] * st["table"].index_select(0, ids[at]).double()
        return dict(out=out)
    # every run of equal ids in the sorted batch, from running sums over its columns
    d_table = (st["table"].double() if c["add"]
               else torch.zeros(c["V"], c["d"], dtype=torch.float64, device=DEV))
    order = ids.argsort(stable=True)
    order = order[ids[order] >= 0]
    if len(order):
        rows, n = ids[order].unique_consecutive(return_counts=True)
        d_table[rows] += st["scale"] * torch.segment_reduce(st["dy"][order].double(), "sum", lengths=n, axis=0)
    return dict(d_table=d_table)


def _exact_rows(st, c, r):
    """The losses and gradient of a block of rows, by differentiation."""
    tau, op = c["tau"], c["op"]
    n = r.stop - r.start
    w = _weight(st)[r].double()
    x = st["x"][r].double().requires_grad_()
    z = torch.log_softmax(x / tau, 1)
    logp = None
    if op.startswith("distill"):
        idx = st["idx"][r].long()
        ok = idx >= 0
        counted = (w != 0) & ok.any(1)
        t = (st["t"][r].double() / tau).masked_fill(~ok, float("-inf"))
        lp = t - torch.logsumexp(t.masked_fill(~ok.any(1, keepdim=True), 0.0), 1, keepdim=True)
        terms = torch.exp(lp).masked_fill(~ok, 0.0) * (lp.masked_fill(~ok, 0.0) - z.gather(1, idx.clamp(min=0)))
        row = tau * tau * terms.masked_fill(~ok, 0.0).sum(1)
    else:
        counted = w != 0
        logp = z[torch.arange(n, device=DEV), st["tok"][r].long()]
        ratio = torch.exp(logp - st["old"][r].double())
        adv = st["adv"][r].double()
        cut = torch.clamp(ratio.detach(), 1 - CLIP[0], 1 + CLIP[1]) * adv
        row = -torch.where(ratio.detach() * adv <= cut, ratio * adv, cut)
        if c["kl"]:
            gap = st["ref"][r].double() - logp
            row = row + c["kl"] * (torch.exp(gap) - 1 - gap)
        logp = torch.where(counted, logp, 0.0).detach()
    row = torch.where(counted, row, 0.0)
    loss = (w * row).sum()
    dx, = torch.autograd.grad(loss, x) if loss.requires_grad else (torch.zeros_like(x),)
    dx = torch.where(counted[:, None], dx * st["grad"].double(), 0.0)
    with torch.no_grad():
        m = x.amax(1)
        s = torch.exp((x - m[:, None]) / tau).sum(1)
        stats = torch.where(counted[:, None], torch.stack([m, s], 1), 0.0)
    return loss.detach(), row.detach(), logp, stats, dx


def _exact_loss(st, c):
    parts = [_exact_rows(st, c, r) for r in _blocks(c["T"], c["V"])]
    loss, row, logp, stats, dx = zip(*parts)
    out = {}
    if not c["op"].endswith("fwd"):
        out["dlogits"] = torch.cat(dx)
    if not c["op"].endswith("bwd"):
        out.update(loss=torch.stack(loss).sum().reshape(1), row_loss=torch.cat(row), stats=torch.cat(stats))
        if logp[0] is not None:
            out["logp"] = torch.cat(logp)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_embed(st, case) if case["op"].startswith("embed") else _exact_loss(st, case)
