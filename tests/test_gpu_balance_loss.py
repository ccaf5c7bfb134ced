"""GPU parity: the router's balance loss and its gradient against the fp64 oracle.

Tolerances.  An fp32 affinity is within 2e-6 of the exact one (the exponential
of the hardware dominates: |l| eps for |l| up to 30, else 1e-6 per unit of
|l|), a probability and a mean of T of them (any order of at most T additions)
within 4e-6 + T 2^-24; the tests keep T 2^-24 below 1e-3 and compare to
4e-6 + (64 + T / 16) 2^-24 relative (a column is summed per wave, then over 16
waves, then over tiles: T / 16 is far above any chain there)."""
import numpy as np
import pytest
import torch

import moe_expert_routing_sqrt_amd as M
from oracle import balance_loss as OL, route as OR

from gpu_util import dev_f32, dev_i32, host, need_gpu

pytestmark = pytest.mark.gpu


def _shape(T, E, k):
    return M.shape(T, 1, E, 1, 1, k, 1, 1)


def _rel(T):
    return 4e-6 + (64 + T / 16) * 2.0 ** -24


def _case(T, E, k, n, ragged, masked, seed, spread=2.0):
    rng = np.random.default_rng(seed)
    L = (rng.normal(size=(T, E)) * spread).astype(np.float32)
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    off = None
    if n > 0:
        off = np.sort(rng.integers(0, T + 1, size=n + 1)).astype(np.int32) if ragged else \
            (np.arange(n + 1) * T // n).astype(np.int32)
    mask = (rng.random(T) > 0.3) if masked else None
    return L, idx, off, mask


def _close(got, ref, rel):
    got, ref = host(got).astype(np.float64), np.asarray(ref, dtype=np.float64)
    assert got.shape == ref.shape
    err = np.abs(got - ref)
    assert (err <= rel * np.abs(ref) + 1e-30).all(), f"worst relative {np.max(err / np.maximum(np.abs(ref), 1e-30))}"


CASES = [  # T, E, k, sequences (0: no offsets), ragged, masked
    (1, 1, 1, 0, False, False), (1, 8, 2, 1, False, False), (3, 3, 3, 0, False, True), (64, 16, 4, 1, False, False),
    (65, 16, 4, 2, False, True), (300, 64, 6, 5, True, True), (257, 256, 8, 0, False, False),
    (1000, 256, 8, 7, True, True), (130, 7, 2, 100, True, False), (64, 5, 1, 64, False, True),
    (500, 100, 16, 3, True, False), (200, 300, 4, 4, True, True), (150, 513, 3, 2, False, False),
    (90, 1024, 16, 3, True, True), (4099, 64, 6, 1, False, False), (40, 24, 3, 1000, True, True),
    (5000, 12, 2, 2, False, True), (700, 256, 16, 40, True, True), (333, 30, 3, 60, True, False),
    (64, 256, 16, 64, False, False), (900, 2, 2, 300, True, True), (3000, 200, 5, 9, True, True),
    (64, 256, 8, 32, True, True), (64, 256, 8, 33, True, True), (65, 16, 2, 1, False, True),
    (63, 127, 7, 3, True, True), (64, 16, 4, 9, True, True),
    (129, 3, 2, 1000, True, True), (30, 3, 2, 1025, True, True), (64, 128, 16, 1, False, False),
    (130, 64, 16, 20, True, True), (30, 7, 2, 1024, True, True)]


@pytest.mark.parametrize("T,E,k,n,ragged,masked", CASES)
def test_loss_and_gradient(T, E, k, n, ragged, masked):
    dev = need_gpu()
    print(f"balance loss T={T} E={E} k={k} n={n} ragged={ragged} masked={masked}", flush=True)
    L, idx, off, mask = _case(T, E, k, n, ragged, masked, T + E)
    sh = _shape(T, E, k)
    offset = np.linspace(-1, 1, E).astype(np.float32) if (T + E) % 2 else None
    Lo = L if offset is None else (L + offset).astype(np.float32)
    ref = OL.forward(Lo, idx, 0.01, off, mask)
    kw = dict(seq_offsets=None if off is None else dev_i32(off, dev),
              token_mask=None if mask is None else torch.from_numpy(mask).to(dev),
              logit_offset=None if offset is None else dev_f32(offset, dev))
    Ld = dev_f32(L, dev)
    loss, counts, prob, dprob = M.balance_loss(sh, Ld, dev_i32(idx, dev), 0.01, **kw)
    torch.cuda.synchronize()
    assert np.array_equal(host(counts), ref[1])
    _close(prob, ref[2], _rel(T))
    _close(dprob, ref[3], 1e-6)
    _close(loss, [ref[0]], _rel(T) + n * 2.0 ** -24)
    # the gradient, from the oracle's dprob; dprob - mean cancels, so the error
    # is relative to the larger of the two
    rng = np.random.default_rng(1)
    extra = rng.normal(size=(T, E)).astype(np.float32) * 1e-3
    dp = ref[3].astype(np.float32)
    for add in (None, extra):
        dl = M.balance_loss_backward(sh, Ld, dev_f32(dp, dev), grad_loss=dev_f32([0.5], dev),
                                     d_extra=None if add is None else dev_f32(add, dev), **kw)
        torch.cuda.synchronize()
        rl = OL.backward(Lo, dp, off, mask, 0.5, add)
        a = OL.affinity(Lo)
        tol = 2e-5 * 0.5 * (dp.max(initial=0.0) / a.sum(1, keepdims=True)) / 2 + 1e-30
        err = np.abs(host(dl) - rl)
        assert (err <= tol + (0 if add is None else 2.0 ** -23 * np.abs(add))).all(), (add is None, (err / tol).max())


def test_from_the_router():
    """Logits, selection and counts of moe_route: the counts of one sequence are
    the column sums of its block counts."""
    dev = need_gpu()
    T, d, E, k = 777, 128, 64, 6
    g = torch.Generator(device=dev).manual_seed(3)
    x = torch.randn(T, d, generator=g, device=dev).to(torch.bfloat16)
    wg = 0.2 * torch.randn(d, E, generator=g, device=dev)
    sh = M.shape(T, d, E, 8, 4, k, 64)
    logits, idx, _, bc = M.route(sh, x, wg, torch.zeros(E, device=dev))
    loss, counts, prob, _ = M.balance_loss(sh, logits, idx, 1.0)
    assert torch.equal(counts[0], bc.sum(0, dtype=torch.int32))
    ref = OL.forward(host(logits), host(idx), 1.0)
    _close(loss, [ref[0]], _rel(T))
    assert abs(float(prob.sum()) - 1) < 1e-5


def test_nothing_counted():
    dev = need_gpu()
    T, E, k = 100, 64, 2
    L, idx, _, _ = _case(T, E, k, 0, False, False, 1)
    sh, Ld, id_ = _shape(T, E, k), dev_f32(L, dev), dev_i32(idx, dev)
    none = torch.zeros(T, dtype=torch.bool, device=dev)
    for kw in (dict(token_mask=none), dict(seq_offsets=dev_i32([50, 50, 50, 50], dev)),
               dict(seq_offsets=dev_i32([100, 100], dev))):
        loss, counts, prob, dprob = M.balance_loss(sh, Ld, id_, 1.0, **kw)
        dl = M.balance_loss_backward(sh, Ld, torch.ones_like(dprob), d_extra=Ld, **kw)
        torch.cuda.synchronize()
        assert float(loss) == 0 and not counts.any() and not prob.any() and not dprob.any()
        assert torch.equal(dl, Ld)
    # no tokens at all
    e = torch.empty(0, E, device=dev)
    loss, counts, prob, dprob = M.balance_loss(_shape(0, E, k), e, torch.empty(0, k, dtype=torch.int32, device=dev),
                                               1.0, seq_offsets=dev_i32([0, 0, 0], dev))
    assert float(loss) == 0 and counts.shape == (2, E) and not counts.any() and not prob.any()
    assert M.balance_loss_backward(_shape(0, E, k), e, dprob, seq_offsets=dev_i32([0, 0, 0], dev)).shape == (0, E)


def test_masked_tokens_may_hold_anything():
    dev = need_gpu()
    for E in (8, 256, 600):
        T, k = 200, 4
        L, idx, off, _ = _case(T, E, k, 3, False, False, 5)
        mask = np.ones(T, dtype=bool)
        mask[::3] = False
        sh, off_d, mask_d = _shape(T, E, k), dev_i32(off, dev), torch.from_numpy(mask).to(dev)
        a = M.balance_loss(sh, dev_f32(L, dev), dev_i32(idx, dev), 0.1, seq_offsets=off_d, token_mask=mask_d)
        ga = M.balance_loss_backward(sh, dev_f32(L, dev), a[3], seq_offsets=off_d, token_mask=mask_d)
        L2, idx2 = L.copy(), idx.copy()
        L2[0::3] = np.nan
        L2[3::6] = np.inf
        L2[6::6] = -np.inf
        idx2[::3] = 2 ** 30
        b = M.balance_loss(sh, dev_f32(L2, dev), dev_i32(idx2, dev), 0.1, seq_offsets=off_d, token_mask=mask_d)
        gb = M.balance_loss_backward(sh, dev_f32(L2, dev), b[3], seq_offsets=off_d, token_mask=mask_d)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a, b)) and torch.equal(ga, gb)
        assert not gb[0::3].any()


def test_extreme_logits():
    """The lowest fp32 value as a mask of experts, rows with no affinity left,
    and large logits: no NaN, and the oracle's probabilities."""
    dev = need_gpu()
    T, E, k = 6, 64, 2
    low = np.finfo(np.float32).min
    L = np.random.default_rng(0).normal(size=(T, E)).astype(np.float32)
    L[1, 5:] = low
    L[2] = low
    L[3] = -60.0
    L[4, ::2] = 80.0
    L[5] = 1e6
    idx = np.tile(np.array([0, 1], dtype=np.int32), (T, 1))
    sh = _shape(T, E, k)
    loss, counts, prob, dprob = M.balance_loss(sh, dev_f32(L, dev), dev_i32(idx, dev), 1.0)
    dl = host(M.balance_loss_backward(sh, dev_f32(L, dev), dprob))
    ref = OL.forward(L, idx, 1.0)
    rl = OL.backward(L, ref[3])
    _close(loss, [ref[0]], 1e-4)  # e^-30 in fp32: 30 units of l times 1e-6 and more
    _close(prob, ref[2], 1e-4)
    assert np.isfinite(dl).all() and not dl[2].any()
    assert (np.abs(dl - rl) <= 1e-4 * np.abs(rl).max(1, keepdims=True) + 1e-30).all()


def test_repeats_and_gradient_against_differences():
    dev = need_gpu()
    T, E, k = 333, 64, 6
    L, idx, off, mask = _case(T, E, k, 4, True, True, 21)
    sh, id_ = _shape(T, E, k), dev_i32(idx, dev)
    kw = dict(seq_offsets=dev_i32(off, dev), token_mask=torch.from_numpy(mask).to(dev))
    Ld = dev_f32(L, dev)
    a = M.balance_loss(sh, Ld, id_, 1.0, **kw)
    for _ in range(5):
        assert all(torch.equal(p, q) for p, q in zip(a, M.balance_loss(sh, Ld, id_, 1.0, **kw)))
    dl = M.balance_loss_backward(sh, Ld, a[3], **kw)
    # the gradient's own direction, large enough to stand clear of the loss's
    # fp32 rounding (about 1e-6 of a loss near 1)
    u = dl / dl.norm()
    h = 2.0
    num = (float(M.balance_loss(sh, Ld + h * u, id_, 1.0, **kw)[0]) -
           float(M.balance_loss(sh, Ld - h * u, id_, 1.0, **kw)[0])) / (2 * h)
    ana = float((dl.double() * u.double()).sum())
    assert abs(num - ana) <= 0.02 * ana + 2e-6, (num, ana)


def test_route_backward_add():
    """dlogits in, the gate's added: dlogits, dx and dw_gate against the oracle's
    gate products on the sum (as the plain call's tolerances)."""
    dev = need_gpu()
    for d, E, xt in ((256, 64, torch.bfloat16), (48, 16, torch.float32)):
        T, k = 200, 4
        g = torch.Generator(device=dev).manual_seed(8)
        sh = M.shape(T, d, E, 4, 2, k, 32)
        x = torch.randn(T, d, generator=g, device=dev).to(xt)
        wg = 0.1 * torch.randn(d, E, generator=g, device=dev)
        logits, idx, _, _ = M.route(sh, x, wg, torch.zeros(E, device=dev))
        dw = torch.randn(T, k, generator=g, device=dev)
        given = 0.1 * torch.randn(T, E, generator=g, device=dev)
        plain, _ = M.route_backward(sh, x, wg, logits, idx, dw, torch.zeros(T, d, device=dev))
        dl, dx = given.clone(), torch.zeros(T, d, device=dev)
        out, dwg = M.route_backward(sh, x, wg, logits, idx, dw, dx, dlogits=dl, add_dlogits=True)
        torch.cuda.synchronize()
        assert out.data_ptr() == dl.data_ptr() and torch.equal(dl, given + plain)
        hd = host(dl).astype(np.float64)
        rx, rw = hd @ host(wg).astype(np.float64).T, host(x).astype(np.float64).T @ hd
        assert np.abs(host(dx) - rx).max() <= 1e-5 * np.abs(rx).max()
        assert np.abs(host(dwg) - rw).max() <= 1e-5 * np.abs(rw).max()


def test_in_a_graph_and_on_another_stream():
    dev = need_gpu()
    T, E, k = 999, 64, 6
    L, idx, off, mask = _case(T, E, k, 5, True, True, 2)
    sh, Ld, id_ = _shape(T, E, k), dev_f32(L, dev), dev_i32(idx, dev)
    kw = dict(seq_offsets=dev_i32(off, dev), token_mask=torch.from_numpy(mask).to(dev))

    def both():
        a = M.balance_loss(sh, Ld, id_, 1.0, **kw)
        return (*a, M.balance_loss_backward(sh, Ld, a[3], **kw))

    ref = both()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = both()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(ref, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for i in range(4):
        Ld.copy_(torch.randn(T, E, device=dev) * 2)
        graph.replay()
        torch.cuda.synchronize()
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)), i


def test_offsets_pass_32_bits():
    """Over 2^31 logits, the counted tokens at the end: as the same tokens alone."""
    dev = need_gpu()
    T, E, k, tail = 2 ** 23 + 64 * 5, 256, 2, 64 * 7
    assert T * E > 2 ** 31
    logits = torch.zeros(T, E, device=dev)
    idx = torch.zeros(T, k, dtype=torch.int32, device=dev)
    logits[-tail:] = torch.randn(tail, E, device=dev)
    idx[-tail:] = torch.randint(0, E, (tail, k), device=dev, dtype=torch.int32)
    off = dev_i32([T - tail, T], dev)
    a = M.balance_loss(_shape(T, E, k), logits, idx, 1.0, seq_offsets=off)
    b = M.balance_loss(_shape(tail, E, k), logits[-tail:].contiguous(), idx[-tail:].contiguous(), 1.0)
    ga = M.balance_loss_backward(_shape(T, E, k), logits, a[3], seq_offsets=off)
    gb = M.balance_loss_backward(_shape(tail, E, k), logits[-tail:].contiguous(), b[3])
    torch.cuda.synchronize()
    assert torch.equal(a[1], b[1]) and torch.equal(a[3], b[3])
    _close(a[0], host(b[0]), _rel(tail))
    _close(a[2], host(b[2]), _rel(tail))
    assert torch.equal(ga[-tail:], gb) and not ga[:-tail].any()
