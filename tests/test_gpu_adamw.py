"""GPU parity: the AdamW step against the oracle's fp32 sequence, bit for bit
(every operation is promised to round once), states and their 8-bit codes
included."""
import numpy as np
import pytest
import torch

import moe_expert_routing_sqrt_amd as M
from oracle import adamw as OA

from gpu_util import host, need_gpu

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
H = dict(lr=1e-2, b1=0.9, b2=0.99, eps=1e-8)


def _bits(a):
    return np.ascontiguousarray(a, dtype=np.float32).view(np.uint32)


def _same(got, want):
    """Equal bits; any NaN equals any NaN."""
    got, want = np.asarray(got, dtype=np.float32), np.asarray(want, dtype=np.float32)
    return np.array_equal(np.isnan(got), np.isnan(want)) and \
        np.array_equal(_bits(got)[~np.isnan(want)], _bits(want)[~np.isnan(want)])


def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def _tensor(a, dt, dev, shift=0):
    """On the GPU at `shift` elements into its storage."""
    t = torch.zeros(a.size + shift, dtype=dt, device=dev)
    t[shift:] = torch.from_numpy(np.ascontiguousarray(a)).to(dev).to(dt)
    return t[shift:]


class Ref:
    """One tensor on the host: what the library holds, by the oracle."""

    def __init__(self, n, p, g, bits, master, seed):
        self.rng = np.random.default_rng(seed)
        self.kind = (p, g, bits, master)
        w = (self.rng.normal(size=n) * 0.05).astype(np.float32)
        self.w = w if p == "f32" or master else _bf16(w)
        self.p = w if p == "f32" else _bf16(w)
        self.m = self.v = np.zeros(n, dtype=np.float32)
        if bits == 8:
            tiles = -(-n // 128)
            self.mc = self.vc = np.zeros(n, dtype=np.uint8)
            self.ms = self.vs = np.ones(tiles, dtype=np.float32)
        self.n = n

    def grad(self):
        g = (self.rng.normal(size=self.n) * np.exp(self.rng.normal(size=self.n) * 2) * 1e-3).astype(np.float32)
        g[self.rng.random(self.n) < 0.1] = 0
        self.g = g if self.kind[1] == "f32" else _bf16(g)
        return self.g

    def step(self, wd, t, scale):
        p, _, bits, master = self.kind
        m, v = self.m, self.v
        if bits == 8:
            r = OA.decode(self.vc, self.vs)
            m, v = OA.decode(self.mc, self.ms), (r * r).astype(np.float32)
        self.w, self.m, self.v, r = OA.step(self.w, self.g, m, v, wd=wd, t=t, scale=scale, **H)
        self.p = self.w if p == "f32" else _bf16(self.w)
        if p == "bf16" and not master:
            self.w = self.p
        if bits == 8:
            self.mc, self.ms = OA.encode(self.m)
            self.vc, self.vs = OA.encode(r)


def _check(opt, i, ref):
    assert _same(host(opt.params[i]).reshape(-1), ref.p), "param"
    if opt.master[i] is not None:
        assert _same(host(opt.master[i]).reshape(-1), ref.w), "master"
    if ref.kind[2] == 8:
        for c, s, rc, rs in ((opt.m[i], opt.m_scale[i], ref.mc, ref.ms), (opt.v[i], opt.v_scale[i], ref.vc, ref.vs)):
            assert _same(host(s), rs), "scale"
            c = host(c.view(torch.uint8))
            nan = (rc & 0x7F) == 0x7F
            assert np.array_equal((c & 0x7F) == 0x7F, nan) and np.array_equal(c[~nan], rc[~nan]), "codes"
    else:
        assert _same(host(opt.m[i]), ref.m) and _same(host(opt.v[i]), ref.v), "states"


KINDS = [(p, g, bits, master) for p, master in (("f32", False), ("bf16", True), ("bf16", False))
         for g in ("f32", "bf16") for bits in (32, 8)]


@pytest.mark.parametrize("p,g,bits,master", KINDS)
def test_steps_bit_for_bit(p, g, bits, master):
    """Several sizes around the 8-element, tile and work-group edges, at odd
    element offsets, three steps with and without a gradient scale."""
    dev = need_gpu()
    print(f"adamw {p} {g} bits={bits} master={master}", flush=True)
    sizes = [1, 7, 8, 127, 128, 129, 1000, 2048, 4097, 0, 20011]
    refs = [Ref(n, p, g, bits, master, 10 + i) for i, n in enumerate(sizes)]
    wd = [0.1 if i % 2 else 0.0 for i in range(len(sizes))]
    params = [_tensor(r.p, DT[p], dev, i % 3) for i, r in enumerate(refs)]
    grads = [_tensor(np.zeros(r.n, np.float32), DT[g], dev, (i + 1) % 2) for i, r in enumerate(refs)]
    ms = [_tensor(r.w, torch.float32, dev, i % 2) for i, r in enumerate(refs)] if master else None
    code = torch.uint8 if bits == 8 else torch.float32
    m = [_tensor(np.zeros(r.n, np.float32), code, dev, i % 5) for i, r in enumerate(refs)]
    v = [_tensor(np.zeros(r.n, np.float32), code, dev, i % 4) for i, r in enumerate(refs)]
    opt = M.AdamW(params, grads, lr=H["lr"], betas=(H["b1"], H["b2"]), eps=H["eps"], weight_decay=wd, master=ms,
                  m=m, v=v)
    for t in (1, 2, 3):
        for gr, r in zip(grads, refs):
            gr.copy_(torch.from_numpy(r.grad()))
        scale = None if t == 2 else 0.37
        opt.step(None if scale is None else torch.tensor([scale], device=dev))
        torch.cuda.synchronize()
        for i, r in enumerate(refs):
            r.step(wd[i], t, scale)
            _check(opt, i, r)
    assert opt.step_count == 3


def test_many_tensors_of_mixed_kinds():
    """More tensors than one launch takes, every kind among them."""
    dev = need_gpu()
    refs = [Ref(50 + 5 * i, *KINDS[i % len(KINDS)], seed=i) for i in range(700)]
    params = [_tensor(r.p, DT[r.kind[0]], dev) for r in refs]
    grads = [_tensor(r.grad(), DT[r.kind[1]], dev) for r in refs]
    master = [_tensor(r.w, torch.float32, dev) if r.kind[3] else None for r in refs]
    code = [torch.uint8 if r.kind[2] == 8 else torch.float32 for r in refs]
    z = lambda: [torch.zeros(r.n, dtype=c, device=dev) for r, c in zip(refs, code)]  # noqa: E731
    opt = M.AdamW(params, grads, lr=H["lr"], betas=(H["b1"], H["b2"]), eps=H["eps"], weight_decay=0.05,
                  master=master, m=z(), v=z())
    opt.step()
    torch.cuda.synchronize()
    for i, r in enumerate(refs):
        r.step(0.05, 1, None)
        _check(opt, i, r)


def test_fresh_states_and_new_masters():
    dev = need_gpu()
    for states in ("f32", "e4m3"):
        r = Ref(3001, "bf16", "f32", 8 if states == "e4m3" else 32, True, 3)
        r.w = r.p                                            # "new" masters start at the rounded weights
        p, g = _tensor(r.p, torch.bfloat16, dev).view(-1, 1), _tensor(r.grad(), torch.float32, dev)
        opt = M.AdamW([p], [g], lr=H["lr"], betas=(H["b1"], H["b2"]), eps=H["eps"], weight_decay=0.1, states=states,
                      master="new")
        opt.step()
        torch.cuda.synchronize()
        r.step(0.1, 1, None)
        _check(opt, 0, r)


@pytest.mark.parametrize("bits", [32, 8])
def test_non_finite_gradients_stay_with_their_element(bits):
    """Infinite, NaN, zero, huge and tiny gradients: bit for bit the oracle's, and
    the finite elements of the tile are what they are without them."""
    dev = need_gpu()
    r, clean = Ref(300, "f32", "f32", bits, False, 4), Ref(300, "f32", "f32", bits, False, 4)
    g = r.grad()
    clean.grad()
    bad = [5, 130, 131, 299]
    for x in (g, clean.g):
        x[10], x[11], x[12] = 0.0, 1e-30, 3e-42
    g[bad] = [np.nan, np.inf, -np.inf, 3e38]
    clean.g[bad] = 0.0
    p, gr = _tensor(r.p, torch.float32, dev), _tensor(g, torch.float32, dev)
    opt = M.AdamW([p], [gr], lr=H["lr"], betas=(H["b1"], H["b2"]), eps=H["eps"], weight_decay=0.0,
                  states="e4m3" if bits == 8 else "f32")
    ok = np.ones(300, dtype=bool)
    ok[bad] = False
    if bits == 8:
        ok[256:] = False    # the tile of the finite 3e38 has another scale
    for t in (1, 2):
        opt.step()
        torch.cuda.synchronize()
        r.step(0.0, t, None)
        clean.step(0.0, t, None)
        _check(opt, 0, r)
        assert _same(host(p)[ok], clean.p[ok])


def test_large_tensor_offsets_pass_32_bits():
    """2^31 + 300 elements of bf16 weights and 8-bit states: the last ones are
    updated as a small tensor of the same values is."""
    dev = need_gpu()
    n, tail = 2 ** 31 + 300, 556  # a whole tile starts at n - 556
    assert (n - tail) % 128 == 0
    p = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    g = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    vals = torch.randn(2, tail, device=dev)
    p[n - tail:], g[n - tail:] = vals[0].to(p.dtype), vals[1].to(p.dtype)
    sp, sg = p[n - tail:].clone(), g[n - tail:].clone()
    a = M.AdamW([p], [g], lr=0.01, states="e4m3")
    b = M.AdamW([sp], [sg], lr=0.01, states="e4m3")
    a.step()
    b.step()
    torch.cuda.synchronize()
    assert torch.equal(p[n - tail:], sp) and not p[:n - tail].any()
    assert torch.equal(a.m[0][n - tail:], b.m[0]) and torch.equal(a.v[0][n - tail:], b.v[0])
    assert torch.equal(a.m_scale[0][(n - tail) // 128:], b.m_scale[0])


def test_more_elements_than_a_launch_reaches():
    """Over 2^34 elements, the most 2^32 threads take at 4 each: around the place where the second launch begins
    and at the end they are updated as small tensors of the same values are, and all others are left at zero."""
    dev = need_gpu()
    first, n = 5000, 2 ** 34 + 3000
    if torch.cuda.mem_get_info()[0] < 120 * 2 ** 30:
        pytest.skip("needs 120 GB of GPU memory")
    places = [((2 ** 32 // 256 - 1 - 5) * 1024 - 2048, 4096), (n - 2000, 2000)]  # 5 work-groups go to the first tensor
    places = [(at // 128 * 128, k) for at, k in places]
    small = torch.randn(first, device=dev).to(torch.bfloat16)
    p, g = (torch.zeros(n, dtype=torch.bfloat16, device=dev) for _ in range(2))
    refs = []
    for at, k in places:
        k = min(k, n - at)
        p[at:at + k], g[at:at + k] = torch.randn(k, device=dev).to(p.dtype), torch.randn(k, device=dev).to(p.dtype)
        refs.append((at, k, p[at:at + k].clone(), g[at:at + k].clone()))
    a = M.AdamW([small, p], [small.clone(), g], lr=0.01, states="e4m3")
    b = M.AdamW([r[2] for r in refs], [r[3] for r in refs], lr=0.01, states="e4m3")
    a.step()
    b.step()
    torch.cuda.synchronize()
    end = 0
    for i, (at, k, want, _) in enumerate(refs):
        assert not p[end:at].any() and not a.m[1][end:at].any()
        assert torch.equal(p[at:at + k], want)
        assert torch.equal(a.m[1][at:at + k], b.m[i]) and torch.equal(a.v[1][at:at + k], b.v[i])
        assert torch.equal(a.v_scale[1][at // 128:-(-(at + k) // 128)], b.v_scale[i])
        end = at + k
    assert end == n or not p[end:].any()


def test_on_another_stream_and_in_a_graph():
    """A captured step repeats its own step number on every replay."""
    dev = need_gpu()
    st = torch.cuda.Stream()
    r = Ref(5000, "f32", "f32", 8, False, 6)
    p, g = _tensor(r.p, torch.float32, dev), _tensor(r.grad(), torch.float32, dev)
    opt = M.AdamW([p], [g], lr=H["lr"], betas=(H["b1"], H["b2"]), eps=H["eps"], weight_decay=0.1, states="e4m3")
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        opt.step()
    st.synchronize()
    r.step(0.1, 1, None)
    _check(opt, 0, r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    for i in range(3):
        g.copy_(torch.from_numpy(r.grad()))
        graph.replay()
        torch.cuda.synchronize()
        r.step(0.1, 2, None)
        _check(opt, 0, r)
