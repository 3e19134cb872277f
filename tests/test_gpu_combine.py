"""GPU tests of moe_decode_combine and its gradients against the definition in
include/moe_decode.h, in float64 on the CPU.

Tolerances, u = 2^-24: y is a chain of k fused multiply-adds in FP32, each rounding
once: (k + 1) u of the sum of the terms' magnitudes, then one rounding to the type.
drows is one product and one rounding.  dweights: a lane's chain of at most N / 64 + 8 fused
multiply-adds, 6 steps over the lanes and at most 4 wavefronts: (N / 64 + 20) u of the
sum of magnitudes.
"""
import pytest
import torch

import moe_gate_up_amd as mg

pytestmark = pytest.mark.gpu
U, TINY = 2.0 ** -24, 1.2e-38
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def make(seed, T, k, N, dtype, dev, M=None, missing=0.2):
    """Positions are distinct; rows that no slot names hold NaN."""
    g = torch.Generator().manual_seed(seed)
    M = T * k + 3 if M is None else M
    at = torch.randperm(M, generator=g)[:T * k].view(T, k).to(torch.int32)
    off = torch.rand(T, k, generator=g) < missing
    at = torch.where(off, torch.tensor([-1, M, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)[torch.randint(0, 4, (T, k), generator=g)], at)
    rows = torch.randn(M, N, generator=g).to(dtype)
    named = torch.zeros(M, dtype=torch.bool)
    named[at[~off].long()] = True
    rows[~named] = float("nan")
    w = torch.randn(T, k, generator=g)
    w[off] = float("nan")   # not looked at
    add, dy = torch.randn(T, N, generator=g).to(dtype), torch.randn(T, N, generator=g).to(dtype)
    return [v.to(dev) for v in (rows, at, w, add, dy)], named


def reference(rows, at, w, add, dy):
    rows, at, add, dy = rows.cpu().double(), at.cpu().long(), None if add is None else add.cpu().double(), dy.cpu().double()
    T, k = at.shape
    on = (at >= 0) & (at < rows.shape[0])
    w = torch.ones(T, k, dtype=torch.float64) if w is None else w.cpu().double()
    w = torch.where(on, w, torch.zeros_like(w))
    r = torch.where(on[:, :, None], rows[at.clamp(0, rows.shape[0] - 1)], torch.zeros((), dtype=torch.float64))
    y = (r * w[:, :, None]).sum(1) + (0 if add is None else add)
    size = (r * w[:, :, None]).abs().sum(1) + (0 if add is None else add.abs())
    dr = torch.zeros_like(rows)
    dr[at[on]] = (w[:, :, None] * dy[:, None, :])[on]
    prod = r * dy[:, None, :]
    return y, size, dr, prod.sum(2), prod.abs().sum(2)


def half(dtype):
    return torch.finfo(dtype).eps / 2


def check(rows, at, w, add, dy, named):
    (T, k), N, dtype = at.shape, rows.shape[1], rows.dtype
    y = torch.full((T, N), 7.0, dtype=dtype, device=rows.device)
    mg.moe_decode_combine(rows, at, w, y, add=add)
    drows, dw = torch.full_like(rows, 5.0), torch.full((T, k), 5.0, device=rows.device)
    mg.moe_decode_combine_backward(dy, rows, at, w, drows, dw)
    only = torch.full_like(rows, 5.0)
    mg.moe_decode_combine_backward(dy, None, at, w, only, None)
    torch.cuda.synchronize()
    assert torch.equal(only, drows)
    ry, size, rdr, rdw, dsize = reference(rows, at, w, add, dy)
    h = half(dtype) if dtype != torch.float32 else 0.0
    small = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    assert bool(((y.cpu().double() - ry).abs() <= (k + 1) * U * size + h * (ry.abs() + (k + 1) * U * size) + small).all())
    assert bool((drows.cpu()[~named] == 5.0).all())
    d = drows.cpu().double()[named]
    assert bool(((d - rdr[named]).abs() <= (U + half(dtype)) * rdr[named].abs() * (1 + U) + small).all())
    assert bool(((dw.cpu().double() - rdw).abs() <= (N / 64 + 20) * U * dsize + TINY).all())


SHAPES = [(1, 1, 1), (1, 8, 2048), (3, 2, 7), (5, 3, 8), (4, 9, 129), (7, 64, 33), (33, 8, 2048), (6, 6, 1000), (2, 17, 4100), (130, 4, 512), (3, 8, 9001)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_against_the_definition(dev, shape, dtype):
    T, k, N = shape
    print(f"combine {shape} {dtype}", flush=True)
    (rows, at, w, add, dy), named = make(T + k + N, T, k, N, dtype, dev)
    check(rows, at, w, add, dy, named)
    check(rows, at, w, None, dy, named)
    check(rows, at, None, add, dy, named)


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_alignment_and_in_place(dev, dtype):
    T, k, N = 20, 5, 200
    (rows, at, w, add, dy), named = make(9, T, k, N, dtype, dev)
    y = torch.empty(T, N, dtype=dtype, device=dev)
    mg.moe_decode_combine(rows, at, w, y, add=add)
    dr, dw = torch.zeros_like(rows), torch.empty(T, k, device=dev)
    mg.moe_decode_combine_backward(dy, rows, at, w, dr, dw)
    for pad, off in ((8, 0), (3, 1), (0, 3)):
        def wide(t):
            b = torch.full((t.shape[0], N + pad + off), 2.0, dtype=dtype, device=dev)
            b[:, off:off + N] = t
            return b, b[:, off:off + N]
        (_, r2), (ab, a2), (_, d2) = wide(rows), wide(add), wide(dy)
        yb, y2 = wide(torch.zeros_like(y))
        mg.moe_decode_combine(r2, at, w, y2, add=a2)
        assert torch.equal(y2, y)
        mg.moe_decode_combine(r2, at, w, a2, add=a2)   # onto what is added
        assert torch.equal(a2, y)
        db, dr2 = wide(torch.zeros_like(rows))
        dw2 = torch.empty_like(dw)
        mg.moe_decode_combine_backward(d2, r2, at, w, dr2, dw2)
        assert torch.equal(dr2, dr) and torch.equal(dw2, dw)
        for b in (yb, ab, db):
            b[:, off:off + N] = 2.0
            assert bool((b == 2.0).all())


def test_no_slot_is_counted_and_infinities(dev):
    (rows, at, w, add, dy), named = make(10, 6, 4, 64, torch.bfloat16, dev, missing=0.0)
    at[2] = -1
    rows[int(at[3, 1]), 5] = float("inf")
    rows[int(at[4, 0]), 6] = float("nan")
    y = torch.empty_like(add)
    mg.moe_decode_combine(rows, at, w, y, add=add)
    assert torch.equal(y[2], add[2])
    assert bool(torch.isinf(y[3, 5])) and bool(torch.isnan(y[4, 6])) and int((~torch.isfinite(y)).sum()) == 2
    mg.moe_decode_combine(rows, at, w, y)
    assert bool((y[2] == 0).all())


def test_gradient_against_differences(dev):
    """y is linear in rows and in weights: f(x + 1) - f(x) is the derivative, in float64 of the definition."""
    (rows, at, w, add, dy), named = make(11, 4, 3, 16, torch.float32, dev)
    drows, dw = torch.zeros_like(rows), torch.empty(4, 3, device=dev)
    mg.moe_decode_combine_backward(dy, rows, at, w, drows, dw)
    f = lambda r, v: float((reference(r, at, v, add, dy)[0] * dy.cpu().double()).sum())   # noqa: E731
    base = f(rows, w)
    for t, j in ((0, 0), (1, 2), (3, 1)):
        if not 0 <= int(at[t, j]) < rows.shape[0]:
            continue
        v = w.clone()
        v[t, j] += 1
        assert abs(f(rows, v) - base - float(dw[t, j])) <= 1e-5
        for n in (0, 15):
            r = rows.clone()
            r[int(at[t, j]), n] += 1
            assert abs(f(r, w) - base - float(drows[int(at[t, j]), n])) <= 1e-5


def test_graph_and_repeat(dev):
    (rows, at, w, add, dy), _ = make(12, 300, 8, 1024, torch.bfloat16, dev)
    y, dr, dw = torch.empty_like(add), torch.zeros_like(rows), torch.empty(300, 8, device=dev)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    mg.moe_decode_combine(rows, at, w, y, add=add, stream=side)
    mg.moe_decode_combine_backward(dy, rows, at, w, dr, dw, stream=side)
    side.synchronize()
    graph, out = torch.cuda.CUDAGraph(), [torch.empty_like(y), torch.zeros_like(dr), torch.empty_like(dw)]
    with torch.cuda.graph(graph):
        mg.moe_decode_combine(rows, at, w, out[0], add=add)
        mg.moe_decode_combine_backward(dy, rows, at, w, out[1], out[2])
    for seed in (1, 2, 3):
        dy.copy_(torch.randn(300, 1024, generator=torch.Generator().manual_seed(seed)))
        add.copy_(dy)
        mg.moe_decode_combine(rows, at, w, y, add=add)
        mg.moe_decode_combine_backward(dy, rows, at, w, dr, dw)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, (y, dr, dw)))


@pytest.mark.parametrize("N", [5, 9, 513, 1025, 2049, 4103])
def test_in_place_where_the_last_columns_are_another_wavefronts(dev, N):
    for dtype in (torch.bfloat16, torch.float32):
        (rows, at, w, add, dy), _ = make(N, 300, 3, N, dtype, dev)
        y = torch.empty_like(add)
        mg.moe_decode_combine(rows, at, w, y, add=add)
        mg.moe_decode_combine(rows, at, w, add, add=add)
        assert torch.equal(add, y)


def test_refusals(dev):
    (rows, at, w, add, dy), _ = make(13, 6, 4, 64, torch.bfloat16, dev)
    y = torch.empty_like(add)
    for args, kw in (((rows, at.long(), w, y), {}), ((rows, at, w.half(), y), {}), ((rows, at, w.t().contiguous(), y), {}), ((rows, at, w, y[:, :63]), {}),
                     ((rows, at, w, y.float()), {}), ((rows, at, w, y), dict(add=add.float())), ((rows, at, w, y), dict(add=add[:5])), ((rows.t(), at, w, y), {})):
        with pytest.raises(ValueError):
            mg.moe_decode_combine(*args, **kw)
    with pytest.raises(mg.MoeDecodeError):
        mg.moe_decode_combine(rows, at, w, rows[:6])
    wide = torch.zeros(7, 64, dtype=torch.bfloat16, device=dev)
    with pytest.raises(mg.MoeDecodeError):   # part of what is added
        mg.moe_decode_combine(rows, at, w, wide[1:], add=wide[:6])
    with pytest.raises(mg.MoeDecodeError):
        mg.moe_decode_combine_backward(dy, rows, at, w, rows, torch.empty(6, 4, device=dev))
    with pytest.raises(ValueError):
        mg.moe_decode_combine_backward(dy, None, at, w, torch.empty_like(rows), torch.empty(6, 4, device=dev))
    mg.moe_decode_combine(rows, at[:0], w[:0], y[:0])
    y.fill_(3.0)
    mg.moe_decode_combine(rows[:0], at, w, y, add=add)   # no rows at all
    assert torch.equal(y, add)
