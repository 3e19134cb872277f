"""GPU tests of moe_decode_route_experts and its gradient against the definition in
include/moe_decode.h, in float64 on the CPU.

Ids are those of 64 bits, exactly (inputs whose choices lie 1e-9 apart among them).

Tolerances, in units of u = 2^-24.  A weight is e^(l - m) / sum: the rounded difference
costs |l - m| u relative, the exponential 2 u.  The sum's terms cost (|l - m| + 3) 2 u of
themselves, on average over the softmax at most (ln E + 3) 2 u = 20 u, the up to 32 + 6
additions 38 u, quotient and factor 2 u: (|l - m| + 62) u, and |l - m| < 40 where a
weight is above 1e-17.  A sigmoid's weight: 6 u, over a sum of up to 64: 80 u.  So 110 u
= 6.6e-6 relative, and FP32's smallest normal number.  The gradient's terms are products of
two or three such values with the caller's gradient and one difference: 3 * 6.6e-6 of
the sum of the terms' magnitudes, and one rounding to the output's type.
"""
import numpy as np
import pytest
import torch

import moe_gate_up_amd as mg

pytestmark = pytest.mark.gpu
REL, TINY = 110 * 2.0 ** -24, 1.2e-38
INF = float("inf")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def scores(l, sigmoid):
    if sigmoid:
        return 1 / (1 + torch.exp(-l))
    m = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(m == -INF, torch.zeros_like(m), m))
    t = e.sum(1, keepdim=True)
    return torch.where(t == 0, torch.zeros_like(e), e / t)


def first(v, n):
    return torch.sort(v, dim=1, descending=True, stable=True).indices[:, :n]


def reference(logits, bias, k, sigmoid, renorm, groups, top, top2, scale):
    """ids and weights in float64 on the CPU."""
    l = logits.detach().cpu().double()
    T, E = l.shape
    s = scores(l, sigmoid)
    out = l == -INF
    c = l if bias is None else torch.where(out, torch.full_like(l, -INF), s + bias.cpu().double())
    if top < groups:
        v = c if bias is not None or not top2 else torch.where(out, torch.full_like(l, -INF), s)
        v = torch.sort(v.view(T, groups, -1), dim=2, descending=True).values
        best = v[:, :, 0]
        if top2 and v.shape[2] > 1:
            best = torch.where(v[:, :, 1] == -INF, best, v[:, :, :2].sum(2))
        keep = torch.zeros(T, groups, dtype=torch.bool).scatter_(1, first(best, top), True).repeat_interleave(E // groups, 1)
        # experts of the groups that stay come first, also those that are ruled out
        order = first(torch.where(keep, c, torch.full_like(c, -INF)), E)
        order = torch.gather(order, 1, first(keep.gather(1, order).double(), E))
        ids = order[:, :k]
    else:
        ids = first(c, k)
    w = s.gather(1, ids)
    if renorm:
        if not sigmoid:   # the same quotients without the small sum
            w = scores(l.gather(1, ids), False)
        else:
            t = w.sum(1, keepdim=True)
            w = torch.where(t == 0, torch.zeros_like(w), w / t)
    return ids, w * scale


def gradient(logits, ids, grad, sigmoid, renorm, scale):
    """dlogits and the magnitudes of its terms in float64."""
    l = logits.detach().cpu().double()
    s = scores(l, sigmoid)
    g = grad.cpu().double() * scale
    p = s.gather(1, ids)
    zero = torch.zeros_like(l)
    if renorm:
        w = scores(l.gather(1, ids), False) if not sigmoid else p / p.sum(1, keepdim=True).clamp_min(1e-300)
        rest = 1 - p if sigmoid else torch.ones_like(p)
        if sigmoid:
            rest = scores(-l.gather(1, ids), True)
        d = w * rest * (g - (g * w).sum(1, keepdim=True))
        size = w * rest * (g.abs() + (g * w).abs().sum(1, keepdim=True))
        return zero.scatter_add(1, ids, d), zero.scatter_add(1, ids, size)
    if sigmoid:
        d = g * p * scores(-l.gather(1, ids), True)
        return zero.scatter_add(1, ids, d), zero.scatter_add(1, ids, d.abs())
    dot = (g * p).sum(1, keepdim=True)
    ds = zero.scatter_add(1, ids, g)
    return s * (ds - dot), s * (ds.abs() + (g * p).abs().sum(1, keepdim=True))


def run(logits, bias, k, sigmoid, renorm, groups, top, top2, scale, grad=None):
    T = logits.shape[0]
    ids = torch.full((T, k), -7, dtype=torch.int32, device=logits.device)
    w = torch.full((T, k), 7.0, device=logits.device)
    mg.moe_decode_route_experts(logits, ids, w, bias=bias, sigmoid=sigmoid, renorm=renorm, groups=groups, top_groups=top,
                                group_top2=top2, scale=scale)
    if grad is None:
        torch.cuda.synchronize()
        return ids, w
    d = torch.full_like(logits, 5.0)
    mg.moe_decode_route_experts_backward(logits, ids, grad, d, sigmoid=sigmoid, renorm=renorm, scale=scale)
    torch.cuda.synchronize()
    return ids, w, d


def check(logits, bias, k, sigmoid, renorm, groups=1, top=1, top2=False, scale=1.0):
    T = logits.shape[0]
    grad = torch.randn(T, k, generator=torch.Generator().manual_seed(T + k)).to(logits.device)
    ids, w, d = run(logits, bias, k, sigmoid, renorm, groups, top, top2, scale, grad)
    rid, rw = reference(logits, bias, k, sigmoid, renorm, groups, top, top2, scale)
    bad = (ids.cpu().long() != rid).any(1).nonzero().flatten()
    assert bad.numel() == 0, (bad[:4], ids[bad[:1]].cpu(), rid[bad[:1]])
    err = (w.cpu().double() - rw).abs() - REL * rw.abs()
    assert bool((err <= TINY).all()), err.max()
    rd, size = gradient(logits, rid, grad, sigmoid, renorm, scale)
    eps = torch.finfo(logits.dtype).eps / 2 if logits.dtype == torch.bfloat16 else 0
    err = (d.cpu().double() - rd).abs() - (3 * REL * size + eps * (rd.abs() + 3 * REL * size))
    assert bool((err <= TINY).all()), err.max()


def make(seed, T, E, dtype, dev):
    g = torch.Generator().manual_seed(seed)
    return (1.5 * torch.randn(T, E, generator=g) + 0.5 * torch.randn(E, generator=g)).to(dtype).to(dev)


SHAPES = [  # T, E, k, groups, top
    (1, 1, 1, 1, 1), (3, 8, 8, 1, 1), (5, 7, 3, 7, 3), (32, 256, 8, 8, 4), (70, 128, 8, 1, 1), (33, 100, 6, 5, 3), (9, 64, 16, 2, 1),
    (17, 72, 4, 9, 2), (13, 255, 16, 15, 4), (21, 256, 17, 16, 9), (11, 250, 64, 2, 1), (7, 1024, 64, 64, 40), (6, 1023, 9, 33, 7),
    (4, 1020, 12, 17, 3), (19, 512, 8, 8, 2), (6, 300, 3, 1, 1), (10, 257, 2, 1, 1), (41, 36, 5, 3, 2), (300, 60, 6, 12, 3), (8, 32, 2, 16, 2),
    (12, 34, 4, 17, 2)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_choices_weights_and_gradient(dev, shape, dtype):
    T, E, k, groups, top = shape
    logits = make(E + T, T, E, dtype, dev)
    bias = (0.1 * torch.randn(E, generator=torch.Generator().manual_seed(E))).to(dev)
    for sigmoid in (False, True):
        for b in (None, bias):
            for renorm in (False, True):
                for top2 in (False, True):
                    print(f"route {shape} {dtype} sigmoid={sigmoid} bias={b is not None} renorm={renorm} top2={top2}", flush=True)
                    check(logits, b, k, sigmoid, renorm, groups, top, top2, 2.5)


def test_many_tokens(dev):
    """Some of these rows' choices differ by less than FP32 can tell."""
    logits = make(3, 40000, 128, torch.float32, dev)
    bias = (0.1 * torch.randn(128, generator=torch.Generator().manual_seed(3))).to(dev)
    check(logits, bias, 8, True, True, 8, 4, True, 2.5)
    check(logits, bias, 8, False, True)
    check(logits, torch.zeros(128, device=dev), 8, True, True, 8, 4, True)
    check(logits.to(torch.bfloat16), torch.zeros(128, device=dev), 8, False, False)


@pytest.mark.parametrize("E", [64, 512])
def test_choices_that_only_64_bits_tell(dev, E):
    """Experts whose score + bias lie about 1e-8 apart, equal in FP32."""
    g = torch.Generator().manual_seed(E)
    bias = (0.2 * torch.randn(E, generator=g)).float()
    l = torch.randn(60, E, generator=g)
    for sigmoid in (True,):
        c = torch.sigmoid(l.double()) + bias.double()
        for t in range(60):
            a, b = c[t].topk(9).indices[torch.tensor([7, 8])].tolist()   # the border of the choice
            s = float(c[t, a] - bias[b].double())
            if 0.05 < s < 0.95:
                l[t, b] = float(np.log(s / (1 - s)))
        check(l.to(dev), bias.to(dev), 8, True, True)
    near = torch.sort(torch.sigmoid(l.double()) + bias.double(), dim=1, descending=True).values
    assert int(((near[:, 7] - near[:, 8]).abs() < 1e-7).sum()) > 30


def test_equal_choices_take_the_lowest(dev):
    E = 48
    l = torch.zeros(6, E)
    l[1] = 3.0
    l[2, ::2] = 1.0
    l[3, 20:] = 40.0     # a sigmoid of 1 in 64 bits
    l[3, 30:] = 41.0
    l[4] = torch.arange(E) // 4
    l[5, 7] = -0.0
    for bias in (None, torch.zeros(E), torch.full((E,), 0.25)):
        for sigmoid in (False, True):
            for top2 in (False, True):
                b = None if bias is None else bias.to(dev)
                check(l.to(dev), b, 7, sigmoid, True)
                check(l.to(dev), b, 7, sigmoid, False, 4, 2, top2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_experts_ruled_out(dev, dtype):
    """-inf and the type's lowest value, up to rows of nothing else."""
    E, k = 64, 6
    l = make(5, 12, E, dtype, dev)
    l[0, 10:] = -INF
    l[1, 3:] = -INF            # fewer than k are left
    l[2] = -INF
    l[3] = torch.finfo(dtype).min
    l[4, :60] = torch.finfo(dtype).min
    l[5, ::2] = -INF
    l[6, 16:] = -INF           # whole groups
    l[7, 1:] = -INF
    l[8, 8:] = -INF
    l[8, 9] = 0
    bias = (0.1 * torch.randn(E, generator=torch.Generator().manual_seed(1))).to(dev)
    for b in (None, bias):
        for sigmoid in (False, True):
            for renorm in (False, True):
                check(l, b, k, sigmoid, renorm)
                for top2 in (False, True):
                    check(l, b, k, sigmoid, renorm, 8, 3, top2)


def test_large_logits_and_biases(dev):
    l = make(8, 40, 96, torch.float32, dev) * 30
    bias = (0.1 * torch.randn(96, generator=torch.Generator().manual_seed(2))).to(dev)
    for b in (None, bias, bias * 1e6, bias * 1e-6):
        for sigmoid in (False, True):
            ids, w = run(l, b, 8, sigmoid, True, 4, 2, False, 1.0)
            rid, rw = reference(l, b, 8, sigmoid, True, 4, 2, False, 1.0)
            assert torch.equal(ids.cpu().long(), rid)
            # |l - m| up to 300 costs that many u
            assert bool(((w.cpu().double() - rw).abs() <= 5 * REL * rw + TINY).all())


def test_not_finite_logits_keep_ids_in_range(dev):
    for E, k in ((64, 8), (300, 20)):
        l = make(9, 30, E, torch.float32, dev)
        l[::3, 5] = float("nan")
        l[1::3, 7] = INF
        l[2::6] = float("nan")
        bias = torch.zeros(E, device=dev)
        for b in (None, bias):
            for sigmoid in (False, True):
                for groups, top in ((1, 1), (4, 2)):
                    ids, _ = run(l, b, k, sigmoid, True, groups, top, True, 1.0)
                    assert int(ids.min()) >= 0 and int(ids.max()) < E
                    assert all(len(set(r)) == k for r in ids.tolist())


def test_strides_and_alignment(dev):
    for dtype in (torch.float32, torch.bfloat16):
        for E, pad, off in ((128, 4, 0), (128, 3, 1), (100, 8, 4), (64, 1, 0)):
            wide = torch.full((50, E + pad + off), 9.0, dtype=dtype, device=dev)
            l = make(E, 50, E, dtype, dev)
            wide[:, off:off + E] = l
            view = wide[:, off:off + E]
            check(view, torch.linspace(-0.1, 0.1, E).to(dev), 4, True, True, 4, 2, True)
            grad = torch.randn(50, 4, device=dev)
            ids, _ = run(l, None, 4, False, False, 1, 1, False, 1.0)
            out = torch.full_like(wide, 3.0)
            mg.moe_decode_route_experts_backward(view, ids, grad, out[:, off:off + E], renorm=False)
            # not bit for bit: a row's columns are dealt out to the lanes by its alignment, so that sums' orders differ
            ref, size = gradient(l, ids.cpu().long(), grad, False, False, 1.0)
            eps = torch.finfo(dtype).eps / 2
            err = (out[:, off:off + E].cpu().double() - ref).abs() - (3 * REL * size + eps * (ref.abs() + 3 * REL * size))
            assert bool((err <= TINY).all())
            out[:, off:off + E] = 3.0
            assert bool((out == 3.0).all())


def test_gradient_against_differences(dev):
    """Of the definition in float64: (f(l + h) - f(l - h)) / 2h, whose own error is h^2 and 1e-16 / h."""
    T, E, k, h = 3, 12, 4, 1e-5
    l = make(11, T, E, torch.float32, dev)
    grad = torch.randn(T, k, generator=torch.Generator().manual_seed(5)).to(dev)
    for sigmoid in (False, True):
        for renorm in (False, True):
            ids, _, d = run(l, None, k, sigmoid, renorm, 1, 1, False, 1.5, grad)
            ids = ids.cpu().long()

            def value(x):
                p = scores(x, sigmoid).gather(1, ids)
                p = p / p.sum(1, keepdim=True) if renorm else p
                return (p * 1.5 * grad.cpu().double()).sum(1)
            for e in range(E):
                step = torch.zeros(T, E, dtype=torch.float64)
                step[:, e] = h
                diff = (value(l.cpu().double() + step) - value(l.cpu().double() - step)) / (2 * h)
                assert bool(((d[:, e].cpu().double() - diff).abs() <= 2e-5).all())


def test_gradient_of_ids_from_elsewhere(dev):
    """Ids out of range contribute nothing, repeated ones add up."""
    l = make(12, 4, 20, torch.float32, dev)
    ids = torch.tensor([[3, 3, 5], [-1, 20, 2], [7, -5, 7], [0, 1, 2]], dtype=torch.int32, device=dev)
    grad = torch.randn(4, 3, generator=torch.Generator().manual_seed(6)).to(dev)
    for sigmoid in (False, True):
        for renorm in (False, True):
            d = torch.full_like(l, 4.0)
            mg.moe_decode_route_experts_backward(l, ids, grad, d, sigmoid=sigmoid, renorm=renorm)
            for t in range(4):
                on = [j for j in range(3) if 0 <= int(ids[t, j]) < 20]
                rd, size = gradient(l[t:t + 1], ids[t:t + 1, on].cpu().long(), grad[t:t + 1, on], sigmoid, renorm, 1.0)
                assert bool(((d[t].cpu().double() - rd[0]).abs() <= 3 * REL * size[0] + TINY).all()), (sigmoid, renorm, t)


def test_graph_stream_and_repeat(dev):
    l = make(13, 500, 128, torch.float32, dev)
    bias = (0.1 * torch.randn(128, generator=torch.Generator().manual_seed(3))).to(dev)
    grad = torch.randn(500, 8, device=dev)
    args = (bias, 8, True, True, 8, 4, True, 2.5)
    ids, w, d = run(l, *args, grad)
    for _ in range(2):
        again = run(l, *args, grad)
        assert all(torch.equal(a, b) for a, b in zip((ids, w, d), again))
    side = torch.cuda.Stream()
    i2, w2 = torch.empty_like(ids), torch.empty_like(w)
    mg.moe_decode_route_experts(l, i2, w2, bias=bias, sigmoid=True, groups=8, top_groups=4, group_top2=True, scale=2.5, stream=side)
    side.synchronize()
    assert torch.equal(i2, ids) and torch.equal(w2, w)
    buf, d2 = l.clone(), torch.empty_like(l)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mg.moe_decode_route_experts(buf, i2, w2, bias=bias, sigmoid=True, groups=8, top_groups=4, group_top2=True, scale=2.5)
        mg.moe_decode_route_experts_backward(buf, i2, grad, d2, sigmoid=True, scale=2.5)
    for seed in (20, 21, 22):
        buf.copy_(make(seed, 500, 128, torch.float32, dev))
        ref = run(buf, *args, grad)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, (i2, w2, d2)))


def test_refusals(dev):
    l = make(14, 10, 16, torch.float32, dev)
    ids, w = torch.empty(10, 2, dtype=torch.int32, device=dev), torch.empty(10, 2, device=dev)
    for bad in (dict(bias=torch.zeros(15, device=dev)), dict(bias=torch.zeros(16, dtype=torch.float64, device=dev))):
        with pytest.raises(ValueError):
            mg.moe_decode_route_experts(l, ids, w, **bad)
    for args in ((l.half(), ids, w), (l.cpu(), ids, w), (l, ids.long(), w), (l, ids[:5], w), (l, ids, w.t().contiguous()), (l.t(), ids, w)):
        with pytest.raises(ValueError):
            mg.moe_decode_route_experts(*args)
    for bad in (dict(groups=3), dict(groups=4, top_groups=5), dict(groups=16, top_groups=1), dict(groups=0), dict(groups=2, top_groups=0)):
        with pytest.raises(mg.MoeDecodeError):
            mg.moe_decode_route_experts(l, ids, w, **bad)
    with pytest.raises(mg.MoeDecodeError):   # in place
        mg.moe_decode_route_experts_backward(l, ids, w, l)
    with pytest.raises(ValueError):
        mg.moe_decode_route_experts_backward(l, ids, w, l.to(torch.bfloat16))
    mg.moe_decode_route_experts(l[:0], ids[:0], w[:0])
