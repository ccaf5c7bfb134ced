"""Layer norm where a call touches more than the package's 256 MB cache (other
loads there), and its parameter gradients to the accuracy of their own chains.

References in fp64 on the GPU, row block by row block.  Tolerances, eps = 2^-24:
the forward's and dx's as in test_gpu_norm.py (64 eps of the largest term of a
row's sum, and the output's rounding).  A parameter gradient's terms are summed
in a lane (the rows that its work-group's slot takes), joined over at most 8
waves, 64 lanes and 512 parts by 16 waves: (rows / (groups * rows at once) + 96)
eps sum|term|, with at least 256 work-groups (or one for every row) that take at
least one row at once."""
import pytest
import torch

import moe_expert_routing_sqrt_amd as M

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ROUND = {"f32": 2.0 ** -23, "bf16": 2.0 ** -8}


def _rows(g, rows, d, dt, dev, offset=0.5):
    t = torch.empty(rows, d, dtype=dt, device=dev)
    for at in range(0, rows, 8192):
        n = min(8192, rows - at)
        t[at:at + n] = torch.randn(n, d, generator=g, device=dev) + offset
    return t


def _blocks(rows, d):
    step = max(1, (1 << 25) // d)
    return [slice(at, min(rows, at + step)) for at in range(0, rows, step)]


def _within(got, ref, tol, what):
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()}"


# rows, d, x, y, residual; each over 256 MB: one piece a lane (d <= 2048), two, and
# rows that share a wave
@pytest.mark.parametrize("rows,d,xt,yt,res", [
    (30000, 2048, "bf16", "bf16", True), (40001, 1017, "f32", "bf16", True), (20000, 2000, "f32", "f32", False),
    (70000, 1024, "bf16", "f32", False), (6000, 7168, "bf16", "bf16", True), (3001, 8191, "f32", "f32", True),
    (5000, 8200, "bf16", "f32", True), (300000, 128, "f32", "f32", True), (400000, 96, "bf16", "bf16", True)])
def test_forward_past_the_cache(rows, d, xt, yt, res):
    dev = need_gpu()
    print(f"norm forward {rows}x{d} {xt}->{yt} res={res}", flush=True)
    size = {"f32": 4, "bf16": 2}
    assert rows * d * (size[xt] * (3 if res else 1) + size[yt]) > 256 * 2 ** 20
    g = torch.Generator(device=dev).manual_seed(rows + d)
    x = _rows(g, rows, d, DT[xt], dev)
    r = _rows(g, rows, d, DT[xt], dev, 0.0) if res else None
    w, b = 1 + 0.2 * torch.randn(d, generator=g, device=dev), 0.2 * torch.randn(d, generator=g, device=dev)
    y, s, mean, rstd = M.layer_norm(x, w, b, residual=r, y_dtype=DT[yt])
    torch.cuda.synchronize()
    for k in _blocks(rows, d):
        want = x[k] if r is None else (x[k].float() + r[k].float()).to(DT[xt])
        assert torch.equal(s[k], want)
        h = want.double()
        rm = h.mean(1, keepdim=True)
        rr = 1 / torch.sqrt(((h - rm) ** 2).mean(1, keepdim=True) + 1e-5)
        big = h.abs().amax(1, keepdim=True)
        _within(mean[k][:, None], rm, 64 * EPS * big, "mean")
        _within(rstd[k][:, None], rr, rr * (64 * EPS + (64 * EPS * big * rr) ** 2), "rstd")
        xh = (h - rm) * rr
        ry = xh * w.double() + b.double()
        tol = 64 * EPS * w.double().abs() * (xh.abs() + big * rr) + ROUND[yt] * ry.abs() + 4 * EPS * b.double().abs()
        _within(y[k], ry, tol + 1e-30, "y")


def _backward_ref(dy, x, w, mean, rstd, ds):
    """(dx, its tolerance without the output's rounding) by blocks, and dw, db with their sums of magnitudes."""
    rows, d = x.shape
    sums = [torch.zeros(d, dtype=torch.float64, device=x.device) for _ in range(4)]
    out = []
    for k in _blocks(rows, d):
        gy, r = dy[k].double(), rstd[k].double()[:, None]
        xh = (x[k].double() - mean[k].double()[:, None]) * r
        q = gy * w.double()
        dx = r * (q - q.mean(1, keepdim=True) - xh * (q * xh).mean(1, keepdim=True))
        tol = r * (q.abs() + q.abs().amax(1, keepdim=True) + xh.abs() * (q * xh).abs().amax(1, keepdim=True))
        if ds is not None:
            dx = dx + ds[k].double()
            tol = tol + ds[k].double().abs()
        out.append((k, dx.float(), (64 * EPS * tol + EPS * dx.abs()).float()))
        t = gy * xh
        for a, v in zip(sums, (t, gy, t.abs(), gy.abs())):
            a += v.sum(0)
    return out, sums


def _chain(rows, d):
    """Additions that a parameter gradient's term goes through, at most."""
    pieces = -(-d // 8)
    waves = -(-pieces // (64 * (1 if pieces <= 1024 else 2)))
    lanes = 64
    while waves == 1 and lanes // 2 >= pieces:
        lanes //= 2
    at_once = 8 * 64 // lanes if waves == 1 else 8 // waves if waves <= 4 else 1
    return -(-rows // (min(256, max(1, rows // at_once)) * at_once)) + 96


# the streaming form takes rows of more than four waves; the rest check dw and db
# where rows share work-groups, with one and two rounds of work-groups a CU
@pytest.mark.parametrize("rows,d,gt,xt,ot,res", [
    (6000, 7168, "f32", "bf16", "bf16", True), (5001, 8191, "bf16", "f32", "f32", True),
    (12000, 2050, "f32", "f32", "f32", False), (9000, 4097, "bf16", "bf16", "f32", True),
    (40007, 100, "f32", "bf16", "f32", False), (100003, 17, "f32", "f32", "f32", True),
    (20000, 264, "bf16", "bf16", "bf16", False), (20000, 1024, "f32", "f32", "bf16", True),
    (250000, 256, "f32", "bf16", "bf16", False), (3000, 9001, "f32", "f32", "f32", True),
    (1025, 2050, "bf16", "bf16", "bf16", False), (500, 2, "f32", "f32", "f32", False)])
def test_backward_values(rows, d, gt, xt, ot, res):
    dev = need_gpu()
    print(f"norm backward {rows}x{d} {gt},{xt}->{ot} res={res}", flush=True)
    g = torch.Generator(device=dev).manual_seed(rows + d)
    x, dy = _rows(g, rows, d, DT[xt], dev), _rows(g, rows, d, DT[gt], dev, 0.1)
    ds = _rows(g, rows, d, DT[xt], dev, 0.0) if res else None
    w = 1 + 0.2 * torch.randn(d, generator=g, device=dev)
    mean = torch.randn(rows, generator=g, device=dev) * 0.1 + 0.5
    rstd = 1 + 0.1 * torch.rand(rows, generator=g, device=dev)
    dx, dw, db = M.layer_norm_backward(dy, x, w, mean, rstd, d_sum=ds, dx_dtype=DT[ot])
    torch.cuda.synchronize()
    ref, (rw, rb, aw, ab) = _backward_ref(dy, x, w, mean, rstd, ds)
    for k, want, tol in ref:
        _within(dx[k], want.double(), tol.double() + ROUND[ot] * want.double().abs() + 1e-30, "dx")
    n = _chain(rows, d)
    _within(dw, rw, n * EPS * aw + 1e-30, "dw")
    _within(db, rb, n * EPS * ab + 1e-30, "db")


def test_parameter_gradients_past_32_bits():
    """Over 2^31 elements: dw and db are the sums over all rows, by blocks in fp64."""
    dev = need_gpu()
    rows, d = 299_700, 7168
    assert rows * d > 2 ** 31
    g = torch.Generator(device=dev).manual_seed(1)
    x, dy = _rows(g, rows, d, torch.bfloat16, dev), _rows(g, rows, d, torch.bfloat16, dev, 0.1)
    w = torch.ones(d, device=dev)
    mean = torch.full((rows,), 0.5, device=dev)
    rstd = 1 + 0.1 * torch.rand(rows, generator=g, device=dev)
    dx, dw, db = M.layer_norm_backward(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    sums = [torch.zeros(d, dtype=torch.float64, device=dev) for _ in range(4)]
    for k in _blocks(rows, d):
        gy = dy[k].double()
        t = gy * (x[k].double() - 0.5) * rstd[k].double()[:, None]
        for a, v in zip(sums, (t, gy, t.abs(), gy.abs())):
            a += v.sum(0)
    n = _chain(rows, d)
    _within(dw, sums[0], n * EPS * sums[2], "dw")
    _within(db, sums[1], n * EPS * sums[3], "db")
