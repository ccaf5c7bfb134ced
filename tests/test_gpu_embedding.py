"""GPU parity: the embedding lookup and its gradient against the fp64 oracle.

Tolerances.  U = 2^-24.  A looked-up element is one fp32 product, then rounded to
its type: U |y| + half a step of the type (bf16 2^-8, fp32 nothing more).  A
gradient element sums n terms, in whatever order with at most n - 1 roundings on
a term's way, times scale (one) and where it is added onto old contents one
more, then the type's rounding.  With small integers and a power of two as
scale every operation is exact, and the results are equal."""
import numpy as np
import pytest
import torch

import moe_expert_routing_sqrt_amd as M
from oracle import embedding as OE

from gpu_util import host, need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
STEP = {"f32": U, "bf16": 2.0 ** -8}
TYPES = [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")]


def _at(t, shift):
    """The same contents at an offset of `shift` elements into their storage."""
    s = torch.empty(t.numel() + shift, dtype=t.dtype, device=t.device)
    s[shift:] = t.reshape(-1)
    return s[shift:].view(t.shape)


def _ids(g, T, V, dev, pad=0.2):
    ids = torch.randint(0, V, (T,), generator=g, device=dev)
    # few rows with many tokens, many with none; padding on both sides of the vocabulary
    ids = torch.where(torch.rand(T, generator=g, device=dev) < 0.4, ids % max(1, V // 50), ids)
    out = torch.rand(T, generator=g, device=dev)
    ids = torch.where(out < pad / 2, torch.full_like(ids, -1), ids)
    return torch.where(out > 1 - pad / 2, V + ids, ids).to(torch.int32)


@pytest.mark.parametrize("T,V,d", [(1, 1, 1), (1, 5, 7168), (3, 10, 3), (8, 1000, 7), (33, 50, 9), (5, 64, 2047),
                                   (257, 300, 256), (100, 33, 1001), (64, 20, 20011)])
@pytest.mark.parametrize("xt,yt", TYPES)
def test_lookup(T, V, d, xt, yt):
    dev = need_gpu()
    print(f"embedding {T}x{d} of {V} {xt}->{yt}", flush=True)
    g = torch.Generator(device=dev).manual_seed(T + d)
    ids = _ids(g, T, V, dev)
    table = _at(torch.randn(V, d, generator=g, device=dev).to(DT[xt]), (T + d) % 3)
    out = _at(torch.full((T, d), 7.0, device=dev, dtype=DT[yt]), d % 2)
    assert M.embedding(ids, table, scale=1.7, out=out) is out
    ref = OE.forward(host(ids), host(table), float(np.float32(1.7)))
    assert (np.abs(host(out) - ref) <= (U + STEP[yt]) * np.abs(ref)).all()
    if xt == yt:  # scale 1: a copy
        assert torch.equal(M.embedding(ids, table)[(ids >= 0) & (ids < V)], table[ids[(ids >= 0) & (ids < V)].long()])


def test_lookup_shapes_and_infinities():
    dev = need_gpu()
    table = torch.randn(6, 16, device=dev)
    table[2], table[3, 0] = float("inf"), float("nan")
    ids = torch.tensor([[2, 3, -1], [6, 0, -2 ** 31]], dtype=torch.int32, device=dev)
    out = M.embedding(ids, table, scale=-2.0)
    assert out.shape == (2, 3, 16)
    assert torch.isneginf(out[0, 0]).all() and torch.isnan(out[0, 1, 0])
    assert not out[0, 2].any() and not out[1, 0].any() and not out[1, 2].any()
    assert M.embedding(ids[:0], table).shape == (0, 3, 16)


GRAD = [(0, 7, 5), (1, 1, 1), (1, 3, 8), (5, 4, 3), (64, 8, 33), (65, 2, 40), (130, 1, 17), (200, 3, 2050),
        (1000, 5003, 1001), (777, 40, 259), (3000, 2500, 64), (700, 20, 7168), (9000, 1025, 12), (4096, 262145, 8),
        (2000, 300000, 5)]


@pytest.mark.parametrize("T,V,d", GRAD)
@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("add", [False, True])
def test_gradient(T, V, d, xt, yt, add):
    dev = need_gpu()
    print(f"embedding gradient {T}x{d} of {V} {xt}->{yt} add={add}", flush=True)
    g = torch.Generator(device=dev).manual_seed(T * 3 + d)
    ids = _ids(g, T, V, dev)
    dy = _at(torch.randn(T, d, generator=g, device=dev).to(DT[xt]), (T + d) % 3)
    table = _at(torch.randn(V, d, generator=g, device=dev).to(DT[yt]), d % 2)
    old = table.clone()
    M.embedding_backward(dy, ids, V, scale=0.3, d_table=table, accumulate=add)
    ref, mags, n = OE.backward(host(dy), host(ids), V, float(np.float32(0.3)))
    tol = (n[:, None] + 1) * U * mags
    got = host(table).astype(np.float64)
    if add:
        assert torch.equal(table[torch.from_numpy(n == 0).to(dev)], old[torch.from_numpy(n == 0).to(dev)])
        ref = ref + host(old)
        tol = np.where(n[:, None] > 0, tol + U * np.abs(ref) + STEP[yt] * (np.abs(ref) + tol), 0.0)
    else:
        tol = tol + STEP[yt] * (np.abs(ref) + tol)
    assert (np.abs(got - ref) <= tol).all(), np.abs(got - ref).max()


@pytest.mark.parametrize("T,V,d", [(5000, 3, 64), (20000, 700, 33), (70000, 65536, 16), (262144, 5, 8)])
def test_gradient_is_exact_on_integers(T, V, d):
    """Long runs: their parts and joins lose no token and count none twice."""
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(T)
    ids = _ids(g, T, V, dev)
    dy = torch.randint(-3, 4, (T, d), generator=g, device=dev).float()
    got = M.embedding_backward(dy, ids, V, scale=0.5)
    want = torch.zeros(V + 1, d, device=dev, dtype=torch.float64)
    want.index_add_(0, torch.where((ids >= 0) & (ids < V), ids, V).long(), dy.double())
    assert torch.equal(got.double(), want[:V] * 0.5)
    again = M.embedding_backward(dy, ids, V, scale=0.5, d_table=got, accumulate=True)
    assert torch.equal(again.double(), want[:V])


@pytest.mark.parametrize("run", [1, 63, 64, 65, 66, 127, 128, 129, 191, 192, 193, 300])
@pytest.mark.parametrize("lead", [0, 1, 7, 8, 9, 63])
def test_runs_at_every_border(run, lead):
    """One run of equal ids that starts `lead` positions into the sorted batch, single
    tokens before it and behind it."""
    dev = need_gpu()
    V, d = 400, 6
    ids = torch.cat([torch.arange(lead), torch.full((run,), 200), torch.arange(300, 310)]).to(torch.int32)
    g = torch.Generator().manual_seed(run)
    ids = ids[torch.randperm(len(ids), generator=g)].to(dev)
    dy = torch.randint(-8, 9, (len(ids), d), generator=g).float().to(dev)
    want = torch.zeros(V, d, dtype=torch.float64)
    want.index_add_(0, ids.cpu().long(), dy.cpu().double())
    assert torch.equal(M.embedding_backward(dy, ids, V).cpu().double(), want)


def test_gradient_of_one_id_only_and_of_none():
    dev = need_gpu()
    dy = torch.ones(4097, 20, device=dev, dtype=torch.bfloat16)
    ids = torch.full((4097,), 9, dtype=torch.int32, device=dev)
    got = M.embedding_backward(dy, ids, 10)
    assert (got[9] == 4097).all() and not got[:9].any()
    kept = torch.full((10, 20), 3.0, device=dev)
    assert (M.embedding_backward(dy, ids - 10, 10, d_table=kept, accumulate=True) == 3).all()
    assert not M.embedding_backward(dy, ids + 1, 10).any()
    nan = dy.clone()
    nan[5, 3] = float("nan")
    ids[5] = -1
    assert torch.isfinite(M.embedding_backward(nan, ids, 10)).all()  # a padding token's gradient is not read


def test_gradient_is_the_lookups_by_differences():
    """<d_table, e> = d/dh <dy, embedding(ids, table + h e)>, exact as the lookup is linear."""
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(0)
    ids, V, d = _ids(g, 300, 90, dev), 90, 24
    dy = torch.randint(-4, 5, (300, d), generator=g, device=dev).float()
    table, e = (torch.randint(-4, 5, (V, d), generator=g, device=dev).float() for _ in range(2))
    step = M.embedding(ids, table + e, scale=2.0) - M.embedding(ids, table, scale=2.0)
    assert (step.double() * dy.double()).sum() == (M.embedding_backward(dy, ids, V, scale=2.0).double() * e.double()).sum()


@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float32])
def test_longest_rows(xt):
    """Rows of the largest size, one of them with a long run."""
    dev = need_gpu()
    T, V, d = 90, 3, 1 << 20
    ids = torch.full((T,), 2, dtype=torch.int32, device=dev)
    ids[7], ids[9] = 0, -1
    table = torch.randint(-8, 9, (V, d), device=dev).to(xt)
    out = M.embedding(ids[:10], table, scale=2.0)
    assert torch.equal(out[8], table[2] * 2) and torch.equal(out[7], table[0] * 2) and not out[9].any()
    dy = torch.randint(-1, 2, (T, d), device=dev).to(xt)  # sums of at most 88: exact in bf16
    got = M.embedding_backward(dy, ids, V, dtype=xt)
    rest = torch.ones(T, dtype=torch.bool)
    rest[[7, 9]] = False
    assert torch.equal(got[2].float(), dy[rest.to(dev)].float().sum(0))
    assert torch.equal(got[0], dy[7]) and not got[1].any()


def test_past_32_bit_offsets():
    """Tables and batches of more than 2^32 elements."""
    dev = need_gpu()
    V, d = 600000, 8192  # 4.9 G elements
    table = torch.zeros(V, d, dtype=torch.bfloat16, device=dev)
    ids = torch.tensor([V - 1, 0, 530000, V - 1, V - 2], dtype=torch.int32, device=dev)
    table[ids.long()] = torch.tensor([1, 2, 3, 1, 5], dtype=torch.bfloat16, device=dev)[:, None]
    assert torch.equal(M.embedding(ids, table)[:, 17].float().cpu(), torch.tensor([1.0, 2, 3, 1, 5]))
    dy = torch.ones(5, d, dtype=torch.bfloat16, device=dev)
    M.embedding_backward(dy, ids, V, d_table=table)
    want = torch.zeros(V, device=dev)
    want.index_add_(0, ids.long(), torch.ones(5, device=dev))
    assert torch.equal(table[:, 0].float(), want) and torch.equal(table[:, d - 1].float(), want)
    del table, dy, want
    T, d = 540000, 8192  # a batch of 4.4 G elements
    dy = torch.zeros(T, d, dtype=torch.bfloat16, device=dev)
    dy[T - 1], dy[100] = 4.0, 2.0
    ids = torch.full((T,), -1, dtype=torch.int32, device=dev)
    ids[T - 1], ids[100] = 3, 3
    assert (M.embedding_backward(dy, ids, 8)[3] == 6).all()


def test_equal_bits_on_every_call_streams_and_graphs():
    """The same bits on every call, on another stream, and replayed from a graph with
    new contents, also with two calls at once on two streams."""
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(5)
    T, V, d = 6000, 900, 200
    ids, dy = _ids(g, T, V, dev), torch.randn(T, d, generator=g, device=dev)
    first = M.embedding_backward(dy, ids, V)
    for _ in range(10):
        assert torch.equal(M.embedding_backward(dy, ids, V), first)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for i in range(6):
        with torch.cuda.stream(s1 if i % 2 else s2):
            outs.append(M.embedding_backward(dy, ids, V))
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    table = torch.randn(V, d, generator=g, device=dev)
    out, grad = torch.empty(T, d, device=dev), torch.empty(V, d, device=dev)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        M.embedding(ids, table, scale=3.0, out=out)
        M.embedding_backward(dy, ids, V, d_table=grad)
    for i in range(4):
        ids.copy_(_ids(g, T, V, dev))
        dy.copy_(torch.randn(T, d, generator=g, device=dev))
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, M.embedding(ids, table, scale=3.0))
        assert torch.equal(grad, M.embedding_backward(dy, ids, V))


def test_refusals():
    dev = need_gpu()
    ids, x = torch.zeros(4, dtype=torch.int32, device=dev), torch.zeros(8, 6, device=dev)
    with pytest.raises(ValueError, match="contiguous"):
        M.embedding(ids, x.t())
    with pytest.raises(ValueError, match="out: needs"):
        M.embedding(ids, x, out=x[:3].clone())
    with pytest.raises(TypeError):
        M.embedding(ids, x.half())
    with pytest.raises(TypeError):
        M.embedding(ids, x, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="d_out: needs"):
        M.embedding_backward(x[:2], ids, 8)
    with pytest.raises(ValueError, match="accumulate"):
        M.embedding_backward(x, ids, 8, accumulate=True)
    with pytest.raises(ValueError, match="d_table: needs"):
        M.embedding_backward(x[:4], ids, 9, d_table=x)
    with pytest.raises(M.MoeError):
        M.embedding_backward(x[:4], ids, 8, ws=torch.empty(16, dtype=torch.uint8, device=dev))
    with pytest.raises(M.MoeError):
        M.embedding(ids, x, scale=float("nan"))
