"""GPU tests of moe_decode_balance and moe_decode_balance_backward against the
formulas of include/moe_decode.h in float64.

Tolerances.  A probability is exp(l - m) / sum: the rounded argument of the
exponential costs |l - m| 2^-24 / ln 2 relative (|l - m| <= 25 in these inputs
where p is not negligible: 2.2e-6), the exponential and the sum a few 2^-24; so
a probability is within 4e-6 relative.  Sums over tokens are FP32 over at most
a few hundred terms of one lane (2e-5 at the very most, 4e-6 as measured by
the count of terms here: <= 64 terms x 2^-24) and FP64 beyond.  losses:
1e-5 relative plus, for z, the absolute error of logsumexp (2^-22 (1 + |m|)).
Gradient: each of its terms p F, p dot, p zc z is within 1.2e-5 of its own
magnitude (p twice: as a factor and inside dot), then one rounding to the
output's type (eps / 2 relative), plus FP32's smallest normal number.
Counts and tokens are exact.
"""
import numpy as np
import pytest
import torch

import moe_gate_up_amd as mg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def reference(logits, ids, valid, G, gb=0.0, gz=0.0):
    """losses, counts, tokens, dlogits and the gradient's terms' magnitudes, float64 on the CPU."""
    l = logits.detach().float().cpu().double()
    ids = ids.cpu().long()
    T, E = l.shape
    k, S = ids.shape[1], T // G
    on = torch.ones(T, dtype=torch.bool) if valid is None else valid.cpu().bool()
    l = torch.where(on[:, None], l, torch.zeros_like(l))
    m = l.amax(1, keepdim=True)
    m = torch.where(m == -np.inf, torch.zeros_like(m), m)
    e = torch.exp(l - m)
    s = e.sum(1, keepdim=True)
    p = torch.where(s == 0, torch.zeros_like(e), e / s)
    z = torch.where(s == 0, torch.zeros_like(s), m + torch.log(s))[:, 0]
    counts = torch.zeros(G, E, dtype=torch.int64)
    n = on.view(G, S).sum(1)
    N = int(n.sum())
    group = torch.arange(T) // S
    ok = on[:, None] & (ids >= 0) & (ids < E)
    counts.view(-1).index_add_(0, (group[:, None] * E + ids)[ok], torch.ones(int(ok.sum()), dtype=torch.int64))
    nn = n.clamp_min(1).double()
    f = counts.double() * (E / (k * nn))[:, None]
    share = torch.zeros(G, E, dtype=torch.float64).index_add_(0, group, p * on[:, None])
    losses = torch.stack([((f * share).sum(1) / nn).sum() / G, (z.square() * on).sum() / max(N, 1)])
    F = (gb * f / (G * nn)[:, None])[group]
    dot = (p * F).sum(1, keepdim=True)
    zc = 2 * gz / max(N, 1)
    d = torch.where(on[:, None], p * (F - dot + zc * z[:, None]), torch.zeros_like(p))
    size = torch.where(on[:, None], p * (F.abs() + dot.abs() + abs(zc) * (1 + z.abs())[:, None]), torch.zeros_like(p))
    zmean = float((z.abs() * on).sum() / max(N, 1))
    return losses, counts, torch.cat([n, n.sum()[None]]), d, size, zmean


def inputs(seed, G, S, E, k, dtype, dev, mask, pad=0):
    g = torch.Generator().manual_seed(seed)
    T = G * S
    full = (1.5 * torch.randn(T, E + pad, generator=g) + 0.5 * torch.randn(E + pad, generator=g)).to(dtype)
    full = full.to(dev)
    logits = full[:, :E]
    ids = logits.float().topk(k, dim=1).indices.to(torch.int32)
    valid = None
    if mask == "random":
        valid = (torch.rand(T, generator=g) < 0.6).to(dev)
    elif mask == "one group empty":
        valid = (torch.rand(T, generator=g) < 0.6)
        valid.view(G, S)[G // 2] = False
        valid = valid.to(dev)
    elif mask == "empty":
        valid = torch.zeros(T, dtype=torch.bool, device=dev)
    return logits, ids, valid


def run(logits, ids, valid, G, gb, gz, out=None):
    T, E = logits.shape
    k, dev = ids.shape[1], logits.device
    losses = torch.full((2,), -7.0, device=dev)
    counts = torch.full((G, E), -7, dtype=torch.int32, device=dev)
    tokens = torch.full((G + 1,), -7, dtype=torch.int32, device=dev)
    d = torch.full((T, E), 7.0, dtype=logits.dtype, device=dev) if out is None else out
    mg.moe_decode_balance(logits, ids, losses, counts, tokens, valid=valid)
    mg.moe_decode_balance_backward(logits, counts, tokens, torch.tensor([gb, gz], device=dev), d, k, valid=valid)
    torch.cuda.synchronize()
    return losses, counts, tokens, d


def check(got, ref, dtype, what):
    losses, counts, tokens, d = got
    rl, rc, rt, rd, size, zmean = ref
    assert torch.equal(counts.cpu().long(), rc), what
    assert torch.equal(tokens.cpu().long(), rt), what
    err = (losses.cpu().double() - rl).abs()
    tol = 1e-5 * rl.abs() + torch.tensor([1e-12, 2 * (1 + zmean) ** 2 * 2.0 ** -22])
    print(f"{what}: losses {rl.tolist()}, off {err.tolist()}", flush=True)
    assert torch.all(err <= tol), (what, err, tol)
    derr = (d.cpu().double() - rd).abs()
    dtol = 1.2e-5 * size + torch.finfo(dtype).eps / 2 * (rd.abs() + 1.2e-5 * size) + 1.2e-38
    worst = (derr / dtol).max().item()
    print(f"{what}: gradient uses {worst:.2f} of its bound", flush=True)
    assert worst <= 1, (what, worst)


SHAPES = [
    # G, S, E, k, dtype, mask, columns between the rows
    (1, 1, 1, 1, torch.float32, None, 0), (1, 1, 128, 8, torch.float32, None, 0), (2, 3, 5, 2, torch.float32, "random", 0),
    (1, 64, 128, 8, torch.float32, None, 0), (1, 64, 128, 8, torch.bfloat16, None, 0), (1, 256, 128, 20, torch.float32, "random", 0),
    (1, 257, 96, 17, torch.bfloat16, "random", 0), (1, 200, 700, 8, torch.float32, "random", 0), (1, 129, 1, 1, torch.float32, "empty", 0),
    (3, 37, 100, 6, torch.bfloat16, "random", 0), (3, 37, 100, 6, torch.float32, "random", 4),
    (1, 1000, 256, 8, torch.float32, "random", 3), (4, 513, 65, 64, torch.float32, "one group empty", 0),
    (5, 33, 1000, 8, torch.float32, None, 0), (5, 33, 1000, 8, torch.bfloat16, "random", 24), (2, 150, 1024, 64, torch.float32, None, 0),
    (1, 300, 512, 3, torch.bfloat16, None, 1), (1, 300, 257, 3, torch.float32, "random", 0), (1, 20011, 128, 8, torch.float32, "random", 0),
    (700, 2, 16, 2, torch.float32, "random", 0), (520, 40, 64, 4, torch.bfloat16, "one group empty", 0),
    (2, 31, 12, 12, torch.float32, "empty", 0), (1, 33, 7, 3, torch.bfloat16, "empty", 0),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[str(s) for s in SHAPES])
def test_against_float64(dev, shape):
    G, S, E, k, dtype, mask, pad = shape
    print(f"balance {shape}", flush=True)
    logits, ids, valid = inputs(100 + SHAPES.index(shape), G, S, E, k, dtype, dev, mask, pad)
    ref = reference(logits, ids, valid, G, 0.7, 0.3)
    check(run(logits, ids, valid, G, 0.7, 0.3), ref, dtype, f"balance {shape}")


def test_gradient_against_differences(dev):
    """The gradient's inner product with random directions equals central differences of the float64 losses (the
    counts held): error h^2 f''' (below 1e-6 of the value at h = 1e-3) plus the gradient's own bound."""
    G, S, E, k = 3, 40, 24, 4
    logits, ids, valid = inputs(7, G, S, E, k, torch.float32, dev, "random")
    gb, gz = 0.9, 0.4
    d = run(logits, ids, valid, G, gb, gz)[3].cpu().double()
    l0 = logits.cpu().double()
    on = valid.cpu()
    _, counts, tokens, _, size, _ = reference(logits, ids, valid, G)
    n = tokens[:G].clamp_min(1).double()

    def value(l):
        p = torch.softmax(l, 1)
        z = torch.logsumexp(l, 1)
        f = counts.double() * (E / (k * n))[:, None]
        share = (p * on[:, None]).view(G, S, E).sum(1)
        return gb * ((f * share).sum(1) / n).mean() + gz * (z.square() * on).sum() / tokens[G]

    g = torch.Generator().manual_seed(8)
    for _ in range(5):
        v = torch.randn(l0.shape, generator=g, dtype=torch.float64)
        h = 1e-3
        num = float((value(l0 + h * v) - value(l0 - h * v)) / (2 * h))
        got = float((d * v).sum())
        tol = 1e-5 * float((d.abs() * v.abs()).sum()) + 1e-5 * abs(num)
        print(f"differences {num:.8f} gradient {got:.8f}", flush=True)
        assert abs(num - got) <= tol, (num, got, tol)


def test_ids_out_of_range_and_repeated(dev):
    G, S, E, k = 2, 50, 40, 6
    logits, ids, valid = inputs(11, G, S, E, k, torch.float32, dev, "random")
    g = torch.Generator().manual_seed(12)
    bad = torch.randint(-3, E + 3, ids.shape, generator=g, dtype=torch.int32)
    bad[0] = 2 ** 31 - 1
    bad[1] = -2 ** 31
    bad[2] = 5   # the same expert six times
    bad[-1] = E - 1
    ids = bad.to(dev)
    check(run(logits, ids, valid, G, 1.0, 1.0), reference(logits, ids, valid, G, 1.0, 1.0), torch.float32, "odd ids")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [100, 128, 700])
def test_experts_ruled_out(dev, E, dtype):
    """-inf and the type's lowest value have probability 0; a row of -inf only has no probabilities at all; rows
    that are not valid may hold anything."""
    G, S, k = 2, 45, 5
    logits, ids, _ = inputs(E, G, S, E, k, dtype, dev, None)
    logits = logits.clone()
    logits[::3, ::2] = -np.inf
    logits[1::3, 1::3] = torch.finfo(dtype).min
    logits[7] = -np.inf
    logits[8] = -np.inf
    logits[8, E - 1] = 0.5
    logits[9] = torch.finfo(dtype).min
    valid = torch.ones(G * S, dtype=torch.bool, device=dev)
    for i, v in ((20, np.nan), (21, np.inf), (22, -np.inf), (89, np.nan)):
        logits[i] = v
        valid[i] = False
    logits[23, 5] = np.nan
    valid[23] = False
    # 3.4e38 squared overflows the z loss of row 9, as it does in FP32: its own test below
    logits[9] = torch.tensor(-50.0, dtype=dtype)
    ref = reference(logits, ids, valid, G, 0.5, 0.25)
    assert torch.isfinite(ref[0]).all()
    check(run(logits, ids, valid, G, 0.5, 0.25), ref, dtype, f"ruled out E={E}")


def test_valid_nan_and_inf_show(dev):
    G, S, E, k = 2, 40, 128, 4
    for value in (np.nan, np.inf):
        logits, ids, _ = inputs(3, G, S, E, k, torch.float32, dev, None)
        logits = logits.clone()
        logits[50, 17] = value
        losses, counts, tokens, d = run(logits, ids, None, G, 1.0, 0.0)
        assert torch.isnan(losses).all()
        assert int(counts.sum()) == G * S * k and tokens.tolist() == [S, S, 2 * S]
        rows = torch.isnan(d).any(1).nonzero().flatten().tolist()
        assert rows == [50], rows


def test_zero_gradient_factors(dev):
    logits, ids, _ = inputs(4, 1, 100, 64, 4, torch.float32, dev, None)
    assert torch.count_nonzero(run(logits, ids, None, 1, 0.0, 0.0)[3]) == 0


def test_strided_gradient_leaves_the_rest(dev):
    for pad in (4, 3):
        logits, ids, valid = inputs(5, 1, 60, 48, 4, torch.float32, dev, "random", pad)
        out = torch.full((60, 48 + pad), 9.0, device=dev)
        got = run(logits, ids, valid, 1, 1.0, 1.0, out=out[:, :48])
        assert torch.all(out[:, 48:] == 9.0)
        check(got, reference(logits, ids, valid, 1, 1.0, 1.0), torch.float32, f"strided {pad}")


def test_same_bits_every_time_and_other_streams(dev):
    """Two calls at once, each with its own workspace, on streams of their own; the results are those of one call
    on the current stream, bit for bit."""
    G, S, E, k = 2, 5000, 128, 8
    logits, ids, valid = inputs(6, G, S, E, k, torch.float32, dev, "random")
    first = run(logits, ids, valid, G, 1.0, 1.0)
    streams = [torch.cuda.Stream() for _ in range(2)]
    grad = torch.ones(2, device=dev)
    n = mg.moe_decode_balance_workspace(G * S, E, k, G)
    outs = []
    for _ in range(2):
        outs.append((torch.empty(2, device=dev), torch.empty(G, E, dtype=torch.int32, device=dev),
                     torch.empty(G + 1, dtype=torch.int32, device=dev), torch.empty_like(logits),
                     torch.full((n,), 255, dtype=torch.uint8, device=dev)))
    torch.cuda.synchronize()
    for _ in range(3):
        for s, (lo, co, to, d, ws) in zip(streams, outs):
            mg.moe_decode_balance(logits, ids, lo, co, to, valid=valid, workspace=ws, stream=s)
            mg.moe_decode_balance_backward(logits, co, to, grad, d, k, valid=valid, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(o[:4], first):
            assert torch.equal(a, b)
    with pytest.raises(ValueError):
        mg.moe_decode_balance(logits, ids, *outs[0][:3], valid=valid, stream=streams[0])


def test_captured_step(dev):
    """Loss and gradient captured once and replayed on changed inputs, with eager calls between the replays."""
    G, S, E, k = 2, 300, 100, 6
    logits, ids, valid = inputs(21, G, S, E, k, torch.float32, dev, "random")
    logits = logits.contiguous()
    grad = torch.tensor([0.3, 0.2], device=dev)
    losses, counts = torch.empty(2, device=dev), torch.empty(G, E, dtype=torch.int32, device=dev)
    tokens, d = torch.empty(G + 1, dtype=torch.int32, device=dev), torch.empty_like(logits)

    def step():
        mg.moe_decode_balance(logits, ids, losses, counts, tokens, valid=valid)
        mg.moe_decode_balance_backward(logits, counts, tokens, grad, d, k, valid=valid)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(4):
        l2, i2, v2 = inputs(30 + rep, G, S, E, k, torch.float32, dev, "random")
        logits.copy_(l2)
        ids.copy_(i2)
        valid.copy_(v2)
        want = run(l2, i2, v2, G, 0.3, 0.2)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((losses, counts, tokens, d), want):
            assert torch.equal(a, b), rep


def test_offsets_beyond_32_bits(dev):
    """Row offsets that pass 2^32 elements: three rows a billion elements apart."""
    E, k, ld = 128, 8, (1 << 30)
    big = torch.empty(4 * ld + E, dtype=torch.bfloat16, device=dev)
    logits = big.as_strided((5, E), (ld, 1))
    g = torch.Generator().manual_seed(1)
    logits.copy_((2 * torch.randn(5, E, generator=g)).to(torch.bfloat16).to(dev))
    ids = logits.float().topk(k, dim=1).indices.to(torch.int32)
    got = run(logits, ids, None, 1, 1.0, 1.0)
    check(got, reference(logits, ids, None, 1, 1.0, 1.0), torch.bfloat16, "far rows")


def test_refusals(dev):
    logits, ids, _ = inputs(1, 1, 10, 16, 2, torch.float32, dev, None)
    losses, counts, tokens = torch.empty(2, device=dev), torch.empty(1, 16, dtype=torch.int32, device=dev), torch.empty(2, dtype=torch.int32, device=dev)
    ok = (logits, ids, losses, counts, tokens)
    for i, bad in ((0, logits.half()), (0, logits.t().contiguous().t()), (1, ids.long()), (1, ids[:5]), (2, losses[:1]),
                   (3, counts.float()), (4, tokens[:1]), (4, tokens.long())):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            mg.moe_decode_balance(*args)
    with pytest.raises(ValueError):
        mg.moe_decode_balance(*ok, valid=torch.ones(9, dtype=torch.bool, device=dev))
    with pytest.raises(ValueError):
        mg.moe_decode_balance(*ok, valid=torch.ones(10, device=dev))
    mg.moe_decode_balance(*ok, workspace=torch.empty(16, dtype=torch.uint8, device=dev))   # so few tokens need none
    many = (torch.zeros(300, 16, device=dev), torch.zeros(300, 2, dtype=torch.int32, device=dev)) + ok[2:]
    with pytest.raises(mg.MoeDecodeError):
        mg.moe_decode_balance(*many, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    with pytest.raises(mg.MoeDecodeError):   # 3 groups do not divide 10 tokens
        mg.moe_decode_balance(logits, ids, losses, torch.empty(3, 16, dtype=torch.int32, device=dev),
                              torch.empty(4, dtype=torch.int32, device=dev))
    with pytest.raises(ValueError):
        mg.moe_decode_balance_backward(logits, counts, tokens, losses, logits.to(torch.bfloat16), 2)
    with pytest.raises(mg.MoeDecodeError):   # in place
        mg.moe_decode_balance_backward(logits, counts, tokens, losses, logits, 2)


def test_no_tokens(dev):
    e = torch.empty
    out = [torch.full((2,), 3.0, device=dev), torch.full((1, 16), 3, dtype=torch.int32, device=dev), torch.full((2,), 3, dtype=torch.int32, device=dev)]
    mg.moe_decode_balance(e(0, 16, device=dev), e(0, 2, dtype=torch.int32, device=dev), *out)
    mg.moe_decode_balance_backward(e(0, 16, device=dev), out[1], out[2], out[0], e(0, 16, device=dev), 2)
    torch.cuda.synchronize()
    assert all(torch.all(o == 3) for o in out)


def test_logits_at_the_lowest_value(dev):
    """Experts ruled out with the type's lowest value, and rows of nothing else: a uniform row, whose square of the
    logsumexp passes FP32 and is left to the formula."""
    for dtype in (torch.float32, torch.bfloat16):
        logits, ids, _ = inputs(31, 2, 40, 24, 4, dtype, dev, None)
        low = torch.finfo(dtype).min
        logits[:, 5] = low
        logits[3] = low
        gb, gz = 0.7, 0.0
        losses, counts, tokens, d = run(logits, ids, None, 2, gb, gz)
        ref = reference(logits, ids, None, 2, gb, gz)
        assert torch.equal(counts.cpu().long(), ref[1]) and torch.equal(tokens.cpu().long(), ref[2])
        assert abs(float(losses[0]) - float(ref[0][0])) <= 1e-5 * float(ref[0][0])
        assert float(losses[1]) == np.inf
        bound = 1.2e-5 * ref[4] + torch.finfo(dtype).eps / 2 * (ref[3].abs() + 1.2e-5 * ref[4]) + 1.2e-38
        assert bool(((d.cpu().double() - ref[3]).abs() <= bound).all())
        assert bool((d[torch.arange(80, device=dev) != 3, 5] == 0).all())


def test_a_long_group(dev):
    """More than 512 parts of 32768 tokens.  A part's sums of non-negative FP32 terms are at most 32768 / 32 = 1024
    additions of a lane, 2 between lanes and 8 between wavefronts, each off by 2^-24 at most: 6.2e-5, and the terms
    4e-6 (z's square twice that)."""
    T, E, k = (1 << 24) + 40000, 8, 1
    g = torch.Generator(device=dev).manual_seed(5)
    logits = torch.randn(T, E, generator=g, device=dev).to(torch.bfloat16)
    ids = torch.randint(0, E, (T, k), generator=g, device=dev, dtype=torch.int32)
    losses = torch.zeros(2, device=dev)
    counts = torch.zeros(1, E, dtype=torch.int32, device=dev)
    tokens = torch.zeros(2, dtype=torch.int32, device=dev)
    mg.moe_decode_balance(logits, ids, losses, counts, tokens)
    share, z = torch.zeros(E, dtype=torch.float64, device=dev), 0.0
    for i in range(0, T, 1 << 22):
        l = logits[i:i + (1 << 22)].double()
        share += torch.softmax(l, 1).sum(0)
        z += float(torch.logsumexp(l, 1).square().sum())
    c = torch.bincount(ids.flatten().long(), minlength=E)
    assert torch.equal(counts[0].long(), c) and tokens.tolist() == [T, T]
    want = [float(E / T * (c / T * share).sum()), z / T]
    print(f"a long group: {losses.tolist()} for {want}", flush=True)
    assert abs(float(losses[0]) - want[0]) <= 7e-5 * want[0] and abs(float(losses[1]) - want[1]) <= 7e-5 * want[1]
