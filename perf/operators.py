"""The operators around the MoE layer in a training step, as a benchmark: the
layer norm in front of the layer (with the residual add) and its backward, the
router's balance loss and its gradient, and the AdamW step over the layer's
weights with 32-bit or 8-bit states.

`run` computes them in plain torch (fp32, rounded once at the end), or through
this package's entry points where `own` is true.  `exact` evaluates the same
definitions in fp64, the gradients by automatic differentiation.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
TILE = 128  # elements that share one scale of an 8-bit optimizer state
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
LR, B1, B2, ADAM_EPS, DECAY = 3e-4, 0.9, 0.95, 1e-8, 0.1


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decoding batch's norm: eight tokens, latency is all
        dict(name="norm_fwd_decode", op="norm_fwd", T=8, d=7168, x="bf16", y="bf16", residual=True),
        # a 64-expert layer's norm on an fp32 residual stream
        dict(name="norm_fwd_f32", op="norm_fwd", T=4096, d=2048, x="f32", y="bf16", residual=True),
        # the norm in front of the 256-expert layer, four sequences of 4096
        dict(name="norm_fwd_large", op="norm_fwd", T=16384, d=7168, x="bf16", y="bf16", residual=True),
        # an odd batch and width, no residual: nothing is aligned
        dict(name="norm_bwd_odd", op="norm_bwd", T=1000, d=1001, x="f32", y="f32", dx="f32", residual=False),
        # the backward at the 256-expert layer's size: the layer's fp32 input
        # gradient comes in, the bf16 residual stream's gradient is added
        dict(name="norm_bwd_large", op="norm_bwd", T=16384, d=7168, x="bf16", y="f32", dx="bf16", residual=True),
        # the smallest layer's balance loss, one sequence
        dict(name="balance_fwd_small", op="balance_fwd", T=256, E=16, k=4, seqs=1, ragged=False),
        # the 256-expert router, a loss for each of four sequences
        dict(name="balance_fwd_large", op="balance_fwd", T=16384, E=256, k=8, seqs=4, ragged=False),
        # its gradient, added to the gate's
        dict(name="balance_bwd_large", op="balance_bwd", T=16384, E=256, k=8, seqs=4, ragged=False, add=True),
        # packed sequences of uneven lengths, some empty, with masked tokens and
        # padding at the end
        dict(name="balance_bwd_ragged", op="balance_bwd", T=4096, E=64, k=6, seqs=37, ragged=True, add=False),
        # the smallest layer's weights, all in one step
        dict(name="adamw_small", op="adamw", sizes="1024,65536,32768,4096,2048,64,64", p="f32", g="f32", bits=32,
             master=False),
        # one of eight GPUs' share of a 64-expert layer: bf16 weights with fp32 masters
        dict(name="adamw_experts", op="adamw", sizes="67108864,33554432,8388608,4194304", p="bf16", g="f32", bits=32,
             master=True),
        # four of 256 experts and the shared one, with 8-bit states
        dict(name="adamw8_experts", op="adamw", sizes="117440512,58720256,29360128,14680064", p="bf16", g="f32",
             bits=8, master=True),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "balance_fwd", "balance_bwd", "adamw"])
    if op in ("norm_fwd", "norm_bwd"):
        d = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            d = max(64, d // 64 * 64)
            d = d + 64 if d == 3072 else d
        T = _log(rng, 1, max(1, min(16384, 16384 * 7168 // d)))
        c = dict(op=op, T=T, d=d, x=rng.choice(["f32", "bf16"]), y=rng.choice(["f32", "bf16"]),
                 residual=rng.random() < 0.6)
        if c["x"] == "f32":
            c["T"] = max(1, T // 2)  # the same bytes
        if op == "norm_bwd":
            c["dx"] = rng.choice(["f32", "bf16"])
            c["T"] = max(1, c["T"] // 2) if c["dx"] == "f32" or c["x"] == "f32" else c["T"]
        c["T"] += c["T"] == 3072
        return c
    if op in ("balance_fwd", "balance_bwd"):
        E = rng.choice([8, 16, 24, 32, 48, 64, 96, 128, 160, 192, 256])
        c = dict(op=op, T=_log(rng, 16, 16384), E=E, k=rng.randint(1, 8), seqs=_log(rng, 1, 64),
                 ragged=rng.random() < 0.6)
        if op == "balance_bwd":
            c["add"] = rng.random() < 0.5
        return c
    bits = rng.choice([8, 32])
    total = _log(rng, 10_000, 100_000_000)
    n = rng.randint(1, 40)
    cut = sorted(rng.random() ** 2 for _ in range(n - 1))
    sizes = [max(1, int((b - a) * total)) for a, b in zip([0.0] + cut, cut + [1.0])]
    if rng.random() < 0.5:
        sizes = [max(256, s // 256 * 256) for s in sizes]
    sizes = [s + (s == 3072) for s in sizes]
    p = rng.choice(["f32", "bf16"])
    return dict(op=op, sizes=",".join(map(str, sizes)), p=p, g=rng.choice(["f32", "bf16"]), bits=bits,
                master=p == "bf16" and rng.random() < 0.7)


def _sizes(case):
    return [int(s) for s in case["sizes"].split(",")]


def work(case):
    b = {"f32": 4, "bf16": 2}
    if case["op"] in ("norm_fwd", "norm_bwd"):
        n, x, y, r = case["T"] * case["d"], b[case["x"]], b[case["y"]], case["residual"]
        if case["op"] == "norm_fwd":
            return {"bytes": n * (x + y + (2 * x if r else 0)) + 8 * case["T"] + 8 * case["d"], "flops": 9 * n}
        return {"bytes": n * (x + y + b[case["dx"]] + (x if r else 0)) + 8 * case["T"] + 12 * case["d"],
                "flops": 16 * n}
    if case["op"] in ("balance_fwd", "balance_bwd"):
        n, table = case["T"] * case["E"], case["seqs"] * case["E"]
        if case["op"] == "balance_fwd":
            return {"bytes": 4 * n + 4 * case["T"] * case["k"] + 12 * table, "flops": 30 * n}
        return {"bytes": n * (12 if case["add"] else 8) + 4 * table, "flops": 40 * n}
    n = sum(_sizes(case))
    state = 16 if case["bits"] == 32 else 4 + 16 / TILE
    return {"bytes": n * (b[case["g"]] + state + (8 + b[case["p"]] if case["master"] else 2 * b[case["p"]])),
            "flops": 20 * n}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _stream(g, T, d, dtype):
    """A residual stream: unit rows with an offset and a few loud channels."""
    x = torch.randn(T, d, generator=g, device=DEV)
    x[:, :: max(1, d // 7)] *= 12.0
    return (x + 0.1 * torch.randn(T, 1, generator=g, device=DEV)).to(dtype)


def _prepare_norm(case, g):
    T, d, xt = case["T"], case["d"], DT[case["x"]]
    st = dict(case=case, x=_stream(g, T, d, xt), w=1 + _randn(g, d, scale=0.1), b=_randn(g, d, scale=0.1))
    st["r"] = _randn(g, T, d, scale=0.5, dtype=xt) if case["residual"] else None
    if case["op"] == "norm_bwd":
        x = st["x"].double()
        st["mean"] = x.mean(1).float()
        st["rstd"] = (x.var(1, unbiased=False) + EPS).rsqrt().float()
        st["dy"] = _randn(g, T, d, scale=0.02, dtype=DT[case["y"]])
    return st


def _prepare_balance(case, g):
    T, E, k, n = case["T"], case["E"], case["k"], case["seqs"]
    # logits of unit tokens against a N(0, 0.02) router at d = 7168, and a skew over the experts
    logits = _randn(g, T, E, scale=1.7) + _randn(g, E, scale=0.5)
    idx = logits.topk(k, dim=1).indices.to(torch.int32)
    st = dict(case=case, logits=logits, idx=idx, alpha=1e-2, mask=None)
    if case["ragged"]:
        cuts = torch.randint(0, T + 1, (n + 1,), generator=g, device=DEV).sort().values
        cuts[0] = 0  # some sequences may be empty, and the tokens past the last one are padding
        st["offsets"] = cuts.to(torch.int32)
        st["mask"] = torch.rand(T, generator=g, device=DEV) > 0.1
    else:
        st["offsets"] = (torch.arange(n + 1, device=DEV) * T // n).to(torch.int32)
    if case["op"] == "balance_bwd":
        st["dprob"] = torch.rand(n, E, generator=g, device=DEV) * (2 * 1e-2 / max(1, T))
        st["grad"] = torch.full((1,), 0.5, device=DEV)
        st["given"] = _randn(g, T, E, scale=1e-6) if case["add"] else None
    return st


def _prepare_adamw(case, g):
    # every kind of buffer is one allocation; a tensor starts at a multiple of
    # 256 elements in it, and what lies between is zero
    sizes = _sizes(case)
    starts, at = [], 0
    for s in sizes:
        starts.append(at)
        at += -(-s // 256) * 256
    live = torch.zeros(at, dtype=torch.bool, device=DEV)
    for a, s in zip(starts, sizes):
        live[a:a + s] = True
    w = _randn(g, at, scale=0.02) * live
    grad = _randn(g, at, scale=1e-3) * live
    m = _randn(g, at, scale=2e-4) * live
    v = (torch.rand(at, generator=g, device=DEV) + 0.05) * 1e-6 * live
    st = dict(case=case, p=w.to(DT[case["p"]]), g=grad.to(DT[case["g"]]), t=100,
              w=w if case["master"] else None, scale=torch.full((1,), 0.7, device=DEV))
    if case["bits"] == 32:
        st.update(m=m, v=v, ms=None, vs=None)
    else:
        st["m"], st["ms"] = _to8(m)
        st["v"], st["vs"] = _to8(v.sqrt())
    cut = lambda t, div=1: None if t is None else [t[a // div:a // div - (-s // div)] for a, s in zip(starts, sizes)]  # noqa: E731
    if own:  # the optimizer that a program keeps: it names its tensors once
        import moe_expert_routing_sqrt_amd as M
        st["opt"] = M.AdamW(cut(st["p"]), cut(st["g"]), lr=LR, betas=(B1, B2), eps=ADAM_EPS, weight_decay=DECAY,
                            master=cut(st["w"]), m=cut(st["m"]), v=cut(st["v"]), m_scale=cut(st["ms"], TILE),
                            v_scale=cut(st["vs"], TILE), step_count=st["t"])
    return st


def prepare(case, seed):
    g = _gen(seed)
    if case["op"].startswith("norm"):
        return _prepare_norm(case, g)
    if case["op"].startswith("balance"):
        return _prepare_balance(case, g)
    return _prepare_adamw(case, g)


# ---------------------------------------------------------------- plain forms

def _plain_norm_fwd(st):
    c = st["case"]
    s = st["x"] if st["r"] is None else (st["x"].float() + st["r"].float()).to(st["x"].dtype)
    f = s.float()
    mean = f.mean(1, keepdim=True)
    rstd = torch.rsqrt(((f - mean) * (f - mean)).mean(1, keepdim=True) + EPS)
    y = ((f - mean) * rstd * st["w"] + st["b"]).to(DT[c["y"]])
    out = dict(y=y, mean=mean[:, 0], rstd=rstd[:, 0])
    if st["r"] is not None:
        out["sum"] = s
    return out


def _plain_norm_bwd(st):
    c = st["case"]
    rstd = st["rstd"][:, None]
    xh = (st["x"].float() - st["mean"][:, None]) * rstd
    dy = st["dy"].float()
    q = dy * st["w"]
    dx = rstd * (q - q.mean(1, keepdim=True) - xh * (q * xh).mean(1, keepdim=True))
    if st["r"] is not None:
        dx = dx + st["r"].float()
    return dict(dx=dx.to(DT[c["dx"]]), dw=(dy * xh).sum(0), db=dy.sum(0))


def _affinity(l):
    """sqrt(softplus(l)) in fp32 from exp and log1p."""
    return torch.sqrt(torch.clamp(l, min=0) + torch.log1p(torch.exp(-l.abs())))


def _sequence_of(st):
    """Each token's sequence; n_seq for tokens that do not count."""
    T, n = st["case"]["T"], st["case"]["seqs"]
    s = torch.searchsorted(st["offsets"], torch.arange(T, device=DEV, dtype=torch.int32), right=True) - 1
    return s if st["mask"] is None else torch.where(st["mask"], s, n)


def _plain_balance_fwd(st):
    c = st["case"]
    E, k, n = c["E"], c["k"], c["seqs"]
    seq = _sequence_of(st)
    a = _affinity(st["logits"])
    p = a / a.sum(1, keepdim=True)
    member = (seq == torch.arange(n, device=DEV)[:, None]).float()  # [n, T]
    tokens = member.sum(1, keepdim=True)
    some = torch.clamp(tokens, min=1.0)
    prob = (member @ p) / some
    counts = torch.zeros((n + 1) * E, dtype=torch.int32, device=DEV)
    at = (seq[:, None] * E + st["idx"]).reshape(-1)
    counts.index_add_(0, at, torch.ones_like(at, dtype=torch.int32))
    counts = counts.view(n + 1, E)[:n]
    f = counts * (E / k) / some
    loss = (f * prob).sum() * (st["alpha"] / n)
    return dict(loss=loss.reshape(1), counts=counts, prob=prob, dprob=f / some * (st["alpha"] / n))


def _plain_balance_bwd(st):
    c = st["case"]
    seq = _sequence_of(st)
    l = st["logits"]
    a = _affinity(l)
    total = a.sum(1, keepdim=True)
    table = torch.cat([st["dprob"] * st["grad"], torch.zeros(1, c["E"], device=DEV)])
    dp = table[seq]
    da = (dp - (dp * a).sum(1, keepdim=True) / total) / total
    dl = da * torch.sigmoid(l) / (2 * a)
    return dict(dlogits=dl if st["given"] is None else dl + st["given"])


def _to8(x):
    """Codes and scales of an 8-bit state: e4m3 values of x / 2^j, 2^j the
    smallest power of two that brings the tile's largest magnitude to 448 or less."""
    t = x.reshape(-1, TILE)
    mant, ex = torch.frexp(t.abs().amax(1))
    j = torch.clamp(ex - 9 + (mant > 0.875).to(ex.dtype), min=-100)
    j = torch.where(mant == 0, torch.zeros_like(j), j)
    scale = ((j.to(torch.int32) + 127) << 23).view(torch.float32)
    inv = ((127 - j.to(torch.int32)) << 23).view(torch.float32)
    return (t * inv[:, None]).to(torch.float8_e4m3fn).reshape(-1), scale


def _from8(code, scale):
    return (code.float().reshape(-1, TILE) * scale[:, None]).reshape(-1)


def _adamw_outputs(st):
    return {n: st[n] for n in ("p", "w", "m", "v", "ms", "vs") if st[n] is not None}


def _plain_adamw(st):
    c = st["case"]
    st["t"] += 1
    bc1, bc2 = 1 - B1 ** st["t"], 1 - B2 ** st["t"]
    wide = c["bits"] == 32
    g = st["g"].float() * st["scale"]
    m = st["m"] if wide else _from8(st["m"], st["ms"])
    v = st["v"] if wide else torch.square(_from8(st["v"], st["vs"]))
    w = (st["w"] if c["master"] else st["p"]).float()
    m = m * B1 + g * (1 - B1)
    v = v * B2 + (g * g) * (1 - B2)
    r = torch.sqrt(v)
    w = w * (1 - LR * DECAY) - (m / (r * (1 / math.sqrt(bc2)) + ADAM_EPS)) * (LR / bc1)
    st["p"].copy_(w)
    if c["master"]:
        st["w"].copy_(w)
    if wide:
        st["m"].copy_(m)
        st["v"].copy_(v)
    else:
        for name, x in (("m", m), ("v", r)):
            code, scale = _to8(x)
            st[name].copy_(code)
            st[name + "s"].copy_(scale)
    return _adamw_outputs(st)


# ---------------------------------------------------------------- the framework's operators

def _own_run(st):
    import moe_expert_routing_sqrt_amd as M
    c = st["case"]
    op = c["op"]
    if op == "norm_fwd":
        y, s, mean, rstd = M.layer_norm(st["x"], st["w"], st["b"], residual=st["r"], eps=EPS, y_dtype=DT[c["y"]])
        out = dict(y=y, mean=mean, rstd=rstd)
        if st["r"] is not None:
            out["sum"] = s
        return out
    if op == "norm_bwd":
        dx, dw, db = M.layer_norm_backward(st["dy"], st["x"], st["w"], st["mean"], st["rstd"], d_sum=st["r"],
                                           dx_dtype=DT[c["dx"]])
        return dict(dx=dx, dw=dw, db=db)
    if op == "balance_fwd":
        sh = M.shape(c["T"], 1, c["E"], 1, 1, c["k"], 1, 1)
        loss, counts, prob, dprob = M.balance_loss(sh, st["logits"], st["idx"], st["alpha"],
                                                   seq_offsets=st["offsets"], token_mask=st["mask"])
        return dict(loss=loss, counts=counts, prob=prob, dprob=dprob)
    if op == "balance_bwd":
        sh = M.shape(c["T"], 1, c["E"], 1, 1, c["k"], 1, 1)
        dl = M.balance_loss_backward(sh, st["logits"], st["dprob"], seq_offsets=st["offsets"],
                                     token_mask=st["mask"], grad_loss=st["grad"], d_extra=st["given"])
        return dict(dlogits=dl)
    st["opt"].step(grad_scale=st["scale"])
    return _adamw_outputs(st)


PLAIN = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "balance_fwd": _plain_balance_fwd,
         "balance_bwd": _plain_balance_bwd, "adamw": _plain_adamw}


def run(state):
    return _own_run(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits

def _exact_norm(st, c):
    x = st["x"].double()
    if c["op"] == "norm_fwd":
        s = x if st["r"] is None else (x + st["r"].double()).to(st["x"].dtype).double()
        mean = s.sum(1) / c["d"]
        rstd = ((s * s).sum(1) / c["d"] - mean * mean + EPS) ** -0.5
        y = (s * rstd[:, None] - (mean * rstd)[:, None]) * st["w"].double() + st["b"].double()
        out = dict(y=y, mean=mean, rstd=rstd)
        if st["r"] is not None:
            out["sum"] = x + st["r"].double()
        return out
    # row blocks: the graph holds several fp64 copies of what it differentiates
    w = st["w"].double().requires_grad_()
    b = torch.zeros_like(w).requires_grad_()
    dx, dw, db = [], 0, 0
    for at in range(0, c["T"], 2048):
        rows = slice(at, at + 2048)
        xr = x[rows].requires_grad_()
        mean = xr.mean(1, keepdim=True)
        y = (xr - mean) / torch.sqrt(((xr - mean) ** 2).mean(1, keepdim=True) + EPS) * w + b
        gx, gw, gb = torch.autograd.grad(y, (xr, w, b), st["dy"][rows].double())
        dx.append(gx if st["r"] is None else gx + st["r"][rows].double())
        dw, db = dw + gw, db + gb
    return dict(dx=torch.cat(dx), dw=dw, db=db)


def _exact_balance(st, c):
    T, E, k, n = c["T"], c["E"], c["k"], c["seqs"]
    off = st["offsets"].tolist()
    keep = torch.ones(T, dtype=torch.bool, device=DEV) if st["mask"] is None else st["mask"]
    l = st["logits"].double().requires_grad_()
    a = torch.logaddexp(l, torch.zeros_like(l)) ** 0.5
    p = a / a.sum(1, keepdim=True)
    if c["op"] == "balance_bwd":
        total = torch.zeros((), dtype=torch.float64, device=DEV)
        for s in range(n):
            rows = p[off[s]:off[s + 1]][keep[off[s]:off[s + 1]]]
            total = total + (rows * st["dprob"][s].double()).sum()
        dl, = torch.autograd.grad(total * st["grad"].double()[0], l)
        return dict(dlogits=dl if st["given"] is None else dl + st["given"].double())
    p = p.detach()
    loss, counts, prob, dprob = 0.0, [], [], []
    for s in range(n):
        rows = keep[off[s]:off[s + 1]]
        Ts = int(rows.sum())
        cnt = torch.bincount(st["idx"][off[s]:off[s + 1]][rows].reshape(-1).long(), minlength=E)
        P = p[off[s]:off[s + 1]][rows].sum(0) / max(1, Ts)
        f = cnt.double() * E / (k * max(1, Ts))
        loss = loss + st["alpha"] / n * float((f * P).sum())
        counts.append(cnt)
        prob.append(P)
        dprob.append(f * st["alpha"] / (n * max(1, Ts)))
    return dict(loss=torch.tensor([loss], dtype=torch.float64), counts=torch.stack(counts).to(torch.int32),
                prob=torch.stack(prob), dprob=torch.stack(dprob))


def _exact_adamw(st, c):
    t = st["t"] + 1
    wide = lambda x, s: x.double() if s is None else (x.double().view(-1, TILE) * s.double()[:, None]).view(-1)  # noqa: E731
    g = st["g"].double() * st["scale"].double()
    m = B1 * wide(st["m"], st["ms"]) + (1 - B1) * g
    v = wide(st["v"], st["vs"])
    v = B2 * (v if c["bits"] == 32 else v ** 2) + (1 - B2) * g ** 2
    w = (st["w"] if c["master"] else st["p"]).double()
    w = w - LR * DECAY * w - LR * (m / (1 - B1 ** t)) / ((v / (1 - B2 ** t)) ** 0.5 + ADAM_EPS)
    out = dict(p=w, m=m, v=v)
    if c["master"]:
        out["w"] = w
    if c["bits"] == 8:  # the unrounded values that the codes stand for
        for name, x in (("m", m), ("v", v ** 0.5)):
            tiles = x.view(-1, TILE)
            need = torch.ceil(torch.log2(tiles.abs().amax(1).clamp(min=1e-300) / 448)).clamp(min=-100)
            scale = torch.where(tiles.abs().amax(1) > 0, 2.0 ** need, torch.ones_like(need))
            out[name] = (tiles / scale[:, None]).view(-1)
            out[name + "s"] = scale
    return out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"].startswith("norm"):
        return _exact_norm(st, case)
    if case["op"].startswith("balance"):
        return _exact_balance(st, case)
    return _exact_adamw(st, case)
