"""GPU parity: layer norm and its backward against the fp64 oracle.

Tolerances.  eps = 2^-24.  A row sum takes at most 16 additions in a lane, 6
in the wave and 16 over the waves (d <= 16384; twice the lane's beyond), so a
row's mean is off by at most 64 eps max|s| and its rstd by 64 eps relative
beside what the mean's error adds; y then by
    64 eps |w| (|xh| + max|s| rstd) + the output's rounding.
The backward's row means carry the same 64 eps of their largest term.  A
parameter gradient adds `rows` terms in some order: (rows + 64) eps sum|term|.
A bf16 output is rounded once: 2^-8 of its magnitude covers that."""
import numpy as np
import pytest
import torch

import moe_expert_routing_sqrt_amd as M
from oracle import norm as ON

from gpu_util import host, need_gpu

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ROUND = {"f32": 2.0 ** -23, "bf16": 2.0 ** -8}

SHAPES = [(1, 1), (1, 64), (3, 7), (2, 9), (5, 63), (7, 513), (4, 1000), (33, 1001), (9, 2048), (3, 4099),
          (5, 7168), (2, 16384), (2, 20011), (1, 32768), (1500, 40), (700, 1024), (2051, 264), (384, 333),
          (385, 333), (1025, 2050), (600, 4097), (530, 9001),
          # rows side by side in a wave
          (1000, 64), (777, 128), (500, 5), (4097, 9), (3000, 33), (1234, 256), (100003, 17), (40007, 100)]


def _rows(g, rows, d, dt, dev, offset=0.5, shift=0):
    """Rows at an offset of `shift` elements into their storage."""
    t = (torch.randn(rows * d + shift, generator=g, device=dev) + offset).to(dt)
    return t[shift:].view(rows, d)


def _check(got, ref, tol):
    got, ref = host(got).astype(np.float64), np.asarray(ref)
    assert got.shape == ref.shape
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.abs(got - ref).max()} against {np.max(tol)}"


def _fwd_tol(s, w, xh, rstd, y, kind):
    big = np.abs(s).max(1, keepdims=True) * rstd[:, None]
    return 64 * EPS * np.abs(w) * (np.abs(xh) + big) + ROUND[kind] * np.abs(y) + 1e-30


@pytest.mark.parametrize("rows,d", SHAPES)
@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("res", [False, True])
def test_forward(rows, d, xt, yt, res):
    dev = need_gpu()
    print(f"norm forward {rows}x{d} {xt}->{yt} res={res}", flush=True)
    g = torch.Generator(device=dev).manual_seed(rows * 7 + d)
    shift = (rows + d) % 3                                  # also at odd element offsets
    x = _rows(g, rows, d, DT[xt], dev, shift=shift)
    r = _rows(g, rows, d, DT[xt], dev, shift=1 - shift % 2) if res else None
    w = 1 + 0.2 * torch.randn(d + 1, generator=g, device=dev)[1:]
    b = 0.2 * torch.randn(d, generator=g, device=dev)
    y, s, mean, rstd = M.layer_norm(x, w, b, residual=r, y_dtype=DT[yt])
    torch.cuda.synchronize()
    want = x if r is None else (x.float() + r.float()).to(DT[xt])
    assert torch.equal(s, want)                             # one fp32 add, rounded once
    hs, hw = host(want).astype(np.float64), host(w)
    ry, rm, rr = ON.forward(hs, hw, host(b))
    big = np.abs(hs).max(1)
    _check(mean, rm, 64 * EPS * big + 1e-30)
    # the mean's error enters the squares as its square only
    _check(rstd, rr, rr * (64 * EPS + (64 * EPS * big * rr) ** 2))
    xh = (hs - rm[:, None]) * rr[:, None]
    _check(y, ry, _fwd_tol(hs, hw, xh, rr, ry, yt) + 4 * EPS * np.abs(host(b)))


def test_forward_no_bias_no_stats_given_buffers():
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(2)
    x = _rows(g, 6, 300, torch.bfloat16, dev)
    r = _rows(g, 6, 300, torch.bfloat16, dev)
    w = torch.randn(300, generator=g, device=dev)
    y0, s0, m0, r0 = M.layer_norm(x, w, torch.zeros(300, device=dev), residual=r)
    y1, s1, m1, r1 = M.layer_norm(x, w, residual=r, keep_stats=False)
    assert m1 is None and r1 is None and torch.equal(y0, y1) and torch.equal(s0, s1)
    # the sum in place of x, and of the residual
    xa, ra = x.clone(), r.clone()
    y2, s2, _, _ = M.layer_norm(xa, w, residual=r, sum_out=xa)
    y3, s3, _, _ = M.layer_norm(x, w, residual=ra, sum_out=ra)
    for y, s in ((y2, s2), (y3, s3)):
        assert torch.equal(y, y0) and torch.equal(s, s0)
    assert s2.data_ptr() == xa.data_ptr()


@pytest.mark.parametrize("rows,d", [(1, 1), (900, 5), (300, 513), (700, 1025), (40, 8200), (3, 16385)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_forward_in_place(rows, d, dt):
    """y or the sum over an input; 513, 1025 and 8200: a row's last piece begins a wave or a lane's second piece."""
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(5)
    x, r = _rows(g, rows, d, dt, dev), _rows(g, rows, d, dt, dev)
    w = torch.randn(d, generator=g, device=dev)
    y0, s0, _, _ = M.layer_norm(x, w, residual=r)
    for y, s in ((0, None), (1, None), (None, 0), (None, 1), (0, 1), (1, 0)):
        ab = [x.clone(), r.clone()]
        y1, s1, _, _ = M.layer_norm(ab[0], w, residual=ab[1], y=None if y is None else ab[y],
                                    sum_out=None if s is None else ab[s])
        assert torch.equal(y1, y0) and torch.equal(s1, s0)
    xc = x.clone()
    M.layer_norm(xc, w, y=xc)
    assert torch.equal(xc, M.layer_norm(x, w)[0])
    with pytest.raises(M.MoeError):
        M.layer_norm(x, w, residual=r, y=xc, sum_out=xc)


def test_forward_offset_rows():
    """A mean far above the spread: squares of the centred values keep the variance."""
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(4)
    x = torch.randn(50, 777, generator=g, device=dev) + 1000.0
    w, b = torch.ones(777, device=dev), torch.zeros(777, device=dev)
    y, _, mean, rstd = M.layer_norm(x, w, b)
    hs = host(x).astype(np.float64)
    ry, rm, rr = ON.forward(hs, host(w), host(b))
    xh = (hs - rm[:, None]) * rr[:, None]
    _check(y, ry, _fwd_tol(hs, host(w), xh, rr, ry, "f32"))
    assert np.abs(host(rstd) / rr - 1).max() < 1e-5


def test_forward_special_rows():
    """A constant row gives the bias; a NaN or infinity spoils its own row only."""
    dev = need_gpu()
    d = 1111
    x = torch.randn(5, d, device=dev)
    x[1] = 3.0
    clean = M.layer_norm(x, torch.ones(d, device=dev))[0]
    x[3, 700] = float("nan")
    x[4, 1110] = float("inf")
    b = torch.arange(d, device=dev, dtype=torch.float32)
    y, _, mean, rstd = M.layer_norm(x, torch.ones(d, device=dev), b, eps=1e-4)
    assert torch.equal(y[1], b) and abs(float(rstd[1]) - 100) < 1e-3
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).any()
    y0 = M.layer_norm(x, torch.ones(d, device=dev))[0]
    assert torch.equal(y0[[0, 2]], clean[[0, 2]])


@pytest.mark.parametrize("rows,d", SHAPES)
@pytest.mark.parametrize("gt,xt,ot,res", [("f32", "bf16", "bf16", True), ("f32", "f32", "f32", False),
                                          ("bf16", "bf16", "bf16", False), ("bf16", "f32", "bf16", True),
                                          ("bf16", "bf16", "f32", True), ("f32", "bf16", "f32", False),
                                          ("bf16", "f32", "f32", False), ("f32", "f32", "bf16", True)])
def test_backward(rows, d, gt, xt, ot, res):
    dev = need_gpu()
    print(f"norm backward {rows}x{d} {gt},{xt}->{ot} res={res}", flush=True)
    g = torch.Generator(device=dev).manual_seed(rows * 11 + d)
    x = _rows(g, rows, d, DT[xt], dev, shift=d % 2)
    dy = _rows(g, rows, d, DT[gt], dev, offset=0.1, shift=rows % 3)
    ds = _rows(g, rows, d, DT[xt], dev, offset=0.0, shift=1) if res else None
    w = 1 + 0.2 * torch.randn(d, generator=g, device=dev)
    hx, hy, hw = host(x).astype(np.float64), host(dy).astype(np.float64), host(w).astype(np.float64)
    _, mean, rstd = ON.forward(hx, hw)
    mean32, rstd32 = mean.astype(np.float32), rstd.astype(np.float32)
    dx, dw, db = M.layer_norm_backward(dy, x, w, torch.from_numpy(mean32).to(dev), torch.from_numpy(rstd32).to(dev),
                                       d_sum=ds, dx_dtype=DT[ot])
    torch.cuda.synchronize()
    hs = None if ds is None else host(ds).astype(np.float64)
    rx, rw, rb = ON.backward(hy, hx, hw, mean32, rstd32, hs)
    r = rstd32.astype(np.float64)[:, None]
    xh = (hx - mean32.astype(np.float64)[:, None]) * r
    q = hy * hw
    row = np.abs(q) + np.abs(q).max(1, keepdims=True) + np.abs(xh) * np.abs(q * xh).max(1, keepdims=True)
    tol = 64 * EPS * (r * row + (0 if hs is None else np.abs(hs))) + ROUND[ot] * np.abs(rx) + 1e-30
    _check(dx, rx, tol)
    _check(dw, rw, (rows + 64) * EPS * np.abs(hy * xh).sum(0) + 1e-30)
    _check(db, rb, (rows + 64) * EPS * np.abs(hy).sum(0) + 1e-30)


@pytest.mark.parametrize("rows", [300, 3000])             # the one-launch form, and the one with parts
def test_backward_in_place_no_bias_and_repeat(rows):
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(6)
    x, dy, ds = (_rows(g, rows, 520, torch.bfloat16, dev) for _ in range(3))
    w = torch.randn(520, generator=g, device=dev)
    _, _, mean, rstd = M.layer_norm(x, w)
    dx, dw, db = M.layer_norm_backward(dy, x, w, mean, rstd, d_sum=ds)
    for _ in range(3):                                    # the same bits on every call
        a = M.layer_norm_backward(dy, x, w, mean, rstd, d_sum=ds)
        assert all(torch.equal(p, q) for p, q in zip(a, (dx, dw, db)))
    ex, ew, eb = M.layer_norm_backward(dy, x, w, mean, rstd, d_sum=ds, has_bias=False)
    assert eb is None and torch.equal(ex, dx) and torch.equal(ew, dw)
    dsc = ds.clone()
    got = M.layer_norm_backward(dy, x, w, mean, rstd, d_sum=dsc, dx=dsc)
    assert all(torch.equal(p, q) for p, q in zip(got, (dx, dw, db)))
    for bad in (dy, x):                                   # read while dx is written
        with pytest.raises(M.MoeError):
            M.layer_norm_backward(dy, x, w, mean, rstd, d_sum=ds, dx=bad)


def test_backward_no_rows():
    dev = need_gpu()
    d = 100
    x, s = torch.empty(0, d, device=dev), torch.empty(0, device=dev)
    dw, db = torch.full((d,), 7.0, device=dev), torch.full((d,), 7.0, device=dev)
    M.layer_norm_backward(x, x, torch.ones(d, device=dev), s, s, dw=dw, db=db)
    torch.cuda.synchronize()
    assert not dw.any() and not db.any()
    y, _, mean, _ = M.layer_norm(x, torch.ones(d, device=dev))
    assert y.shape == (0, d) and mean.numel() == 0


def test_gradient_against_differences():
    """Central differences of the GPU's own fp32 forward.  The loss sums n = 40*50
    rounded outputs (error about sqrt(n) eps |y dy|), so a step of 2^-6 leaves a
    relative error near 1e-4; its truncation is of the same size."""
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(9)
    rows, d, h = 40, 50, 2.0 ** -6
    x, dy, u = (torch.randn(rows, d, generator=g, device=dev) for _ in range(3))
    w, b, uw, ub = (torch.randn(d, generator=g, device=dev) for _ in range(4))
    _, _, mean, rstd = M.layer_norm(x, w, b)
    dx, dw, db = M.layer_norm_backward(dy, x, w, mean, rstd)

    def loss(s):
        y = M.layer_norm(x + s * h * u, w + s * h * uw, b + s * h * ub)[0]
        return float((y.double() * dy.double()).sum())

    num = (loss(1) - loss(-1)) / (2 * h)
    ana = float((dx.double() * u.double()).sum() + (dw.double() * uw.double()).sum() + (db.double() * ub.double()).sum())
    scale = float(dy.double().norm())
    assert abs(num - ana) <= 5e-3 * scale, (num, ana, scale)


def test_on_another_stream_and_in_a_graph():
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(12)
    x, r = (_rows(g, 257, 1032, torch.bfloat16, dev) for _ in range(2))
    w, b = torch.randn(1032, generator=g, device=dev), torch.randn(1032, generator=g, device=dev)
    y0, s0, m0, r0 = M.layer_norm(x, w, b, residual=r)
    d0 = M.layer_norm_backward(y0, s0, w, m0, r0, d_sum=r)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        y1, s1, m1, r1 = M.layer_norm(x, w, b, residual=r)
        d1 = M.layer_norm_backward(y1, s1, w, m1, r1, d_sum=r)
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and all(torch.equal(p, q) for p, q in zip(d0, d1))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, s2, m2, r2 = M.layer_norm(x, w, b, residual=r)
        d2 = M.layer_norm_backward(y2, s2, w, m2, r2, d_sum=r)
    for i in range(4):
        x.copy_(torch.randn(257, 1032, generator=g, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        y3, s3, m3, r3 = M.layer_norm(x, w, b, residual=r)
        d3 = M.layer_norm_backward(y3, s3, w, m3, r3, d_sum=r)
        torch.cuda.synchronize()
        assert torch.equal(y2, y3) and all(torch.equal(p, q) for p, q in zip(d2, d3)), i


def test_offsets_pass_32_bits():
    """Over 2^31 elements: the last rows are what the same rows give alone."""
    dev = need_gpu()
    rows, d, tail = 299_700, 7168, 400
    assert rows * d > 2 ** 31
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device=dev)
    x[-tail:] = torch.randn(tail, d, device=dev).to(torch.bfloat16)
    w, b = torch.randn(d, device=dev), torch.randn(d, device=dev)
    y, _, mean, rstd = M.layer_norm(x, w, b)
    sy, _, smean, srstd = M.layer_norm(x[-tail:].contiguous(), w, b)
    assert torch.equal(y[-tail:], sy) and torch.equal(mean[-tail:], smean) and torch.equal(rstd[-tail:], srstd)
    dx, dw, db = M.layer_norm_backward(y, x, w, mean, rstd)
    sx, _, _ = M.layer_norm_backward(sy, x[-tail:].contiguous(), w, smean, srstd)
    torch.cuda.synchronize()
    assert torch.equal(dx[-tail:], sx)
    assert torch.isfinite(dw).all() and torch.isfinite(db).all()
