"""GPU tests of moe_decode_adapters against the definition in include/moe_decode.h,
in float64.

Tolerances, u = 2^-24.  A sum of n products in FP32, in any order, is within n u of the
sum of their magnitudes: v = A x within K u sum |a x|.  v enters the second product as
two 16-bit numbers, within 2^-16 of itself in bf16 (half a step, 2^-8, of a rest that is at
most half a step, 2^-8, of it); in FP16, scaled to the row's largest, within 2^-22 of itself and 2^-38 of
the row's largest.  The second sum has 2 R products: (2 R + 8) u with the factor; base and
result cost 2 u and one rounding to the type.
"""
import pytest
import torch

import moe_gate_up_amd as mg

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def make(seed, M, K, N, R, L, dtype, dev, mixed=True):
    g = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)   # noqa: E731
    if mixed:
        ids = torch.randint(-1, L + 1, (M,), generator=g, device=dev).to(torch.int32)   # -1 and L: none
    else:
        ids = (torch.arange(M, device=dev) * L // M).to(torch.int32)
    return (rnd(M, K).to(dtype), ids, (rnd(L, R, K) * K ** -0.5).to(dtype), rnd(L, N, R).to(dtype),
            0.25 + torch.rand(L, generator=g, device=dev), rnd(M, N).to(dtype))


def check(x, ids, a, b, s, base, y):
    """Row by row of each adapter, on the GPU in float64."""
    L, R, K = a.shape
    dtype = x.dtype
    h, low = torch.finfo(dtype).eps / 2, torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    at = torch.where((ids >= 0) & (ids < L), ids, torch.full_like(ids, -1))
    zero = torch.zeros(x.shape[0], b.shape[1], dtype=torch.float64, device=x.device)
    full = zero if base is None else base.double()
    none = at == -1
    assert torch.equal(y[none], full[none].to(dtype))
    for l in sorted(set(at.tolist()) - {-1}):
        m = (at == l).nonzero().flatten()
        X, A, B, f = x[m].double(), a[l].double(), b[l].double(), float(s[l].double())
        v = X @ A.t().contiguous()
        ev = K * U * (X.abs() @ A.abs().t().contiguous()) + (2.0 ** -16 + (2 * R + 8) * U) * v.abs()
        ev = ev + 2.0 ** -38 * v.abs().amax(1, keepdim=True)
        Bt = B.t().contiguous()
        ref = full[m] + f * (v @ Bt)
        err = f * (ev @ Bt.abs()) + 2 * U * (full[m].abs() + ref.abs())
        bad = (y[m].double() - ref).abs() - (err + h * (ref.abs() + err) + low)
        assert bool((bad <= 0).all()), (l, float(bad.max()))


def run(x, ids, a, b, s, base, **kw):
    y = torch.full((x.shape[0], b.shape[1]), 7.0, dtype=x.dtype, device=x.device)
    mg.moe_decode_adapters(x, ids, a, b, s, y, base=base, **kw)
    torch.cuda.synchronize()
    return y


SHAPES = [  # M, K, N, R, L
    (1, 8, 1, 8, 1), (1, 2048, 4096, 16, 4), (3, 64, 65, 24, 2), (16, 128, 64, 32, 1), (17, 136, 200, 16, 1), (32, 2048, 1000, 16, 64),
    (33, 72, 63, 40, 3), (40, 1000, 129, 64, 5), (64, 512, 300, 128, 7), (100, 320, 77, 8, 1000), (21, 200, 130, 136, 2), (9, 264, 500, 256, 2),
    (384, 96, 80, 16, 33), (385, 96, 80, 16, 33), (1, 4096, 200, 64, 3), (7, 8192, 100, 32, 2), (40, 1024, 300, 256, 4),
    (130, 8192, 64, 24, 5), (600, 264, 1030, 48, 9), (1500, 128, 257, 64, 1), (5000, 64, 100, 8, 1023), (4097, 512, 64, 256, 3)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_against_the_definition(dev, shape, dtype):
    print(f"adapters {shape} {dtype}", flush=True)
    for mixed in (True, False):
        x, ids, a, b, s, base = make(sum(shape), *shape, dtype, dev, mixed)
        check(x, ids, a, b, s, base, run(x, ids, a, b, s, base))
        check(x, ids, a, b, s, None, run(x, ids, a, b, s, None))


@pytest.mark.parametrize("M", [30, 700])
def test_rows_without_an_adapter(dev, M):
    x, ids, a, b, s, base = make(1, M, 128, 150, 16, 4, torch.bfloat16, dev)
    for fill in (-1, 4, 2 ** 31 - 1, -2 ** 31):
        ids.fill_(fill)
        assert torch.equal(run(x, ids, a, b, s, base), base)
        assert bool((run(x, ids, a, b, s, None) == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [50, 800])
def test_strides_and_in_place(dev, M, dtype):
    K, N = 256, 203
    x, ids, a, b, s, base = make(2, M, K, N, 32, 6, dtype, dev)
    y = run(x, ids, a, b, s, base)
    wide = torch.full((M, K + 24), 9.0, dtype=dtype, device=dev)
    wide[:, 8:8 + K] = x
    for pad, off in ((5, 0), (8, 3)):
        bb = torch.full((M, N + pad + off), 2.0, dtype=dtype, device=dev)
        yb = bb.clone()
        bb[:, off:off + N] = base
        mg.moe_decode_adapters(wide[:, 8:8 + K], ids, a, b, s, yb[:, off:off + N], base=bb[:, off:off + N])
        assert torch.equal(yb[:, off:off + N], y)
        view = bb[:, off:off + N]
        mg.moe_decode_adapters(x, ids, a, b, s, view, base=view)   # onto the base
        assert torch.equal(view, y)
        for t in (bb, yb):
            t[:, off:off + N] = 2.0
            assert bool((t == 2.0).all())


def test_fp16_range(dev):
    """Inner values beyond FP16's range and far below it."""
    for scale, back in ((1e3, 1e-4), (1e-3, 1.0)):
        x, ids, a, b, s, base = make(3, 20, 512, 64, 16, 3, torch.float16, dev)
        x, a = (x * (30 if scale > 1 else scale)).half(), (a * scale).half()
        b = (b * back).half()
        check(x, ids, a, b, s, base, run(x, ids, a, b, s, base))


def test_infinities_stay_in_their_rows(dev):
    for dtype in TYPES:
        x, ids, a, b, s, base = make(4, 40, 128, 96, 16, 2, dtype, dev)
        ids = ids.clamp(0, 1)
        clean = run(x, ids, a, b, s, base)
        x[3, 5] = float("nan")
        x[7, 6] = float("inf")
        base[9, 1] = float("inf")
        y = run(x, ids, a, b, s, base)
        assert bool(torch.isnan(y[3]).all()) and not bool(torch.isfinite(y[7]).any()) and bool(torch.isinf(y[9, 1]))
        keep = [m for m in range(40) if m not in (3, 7, 9)]
        assert torch.equal(y[keep], clean[keep])


def test_graph_stream_workspace_and_repeat(dev):
    for M in (64, 900):
        x, ids, a, b, s, base = make(5, M, 256, 320, 16, 9, torch.bfloat16, dev)
        need = mg.moe_decode_adapters_workspace(M, 256, 320, 16, 9)
        assert (need > 0) == (M == 900)   # without one and with
        ws = torch.full((max(need, 256),), 0xAB, dtype=torch.uint8, device=dev)
        y = run(x, ids, a, b, s, base)
        assert torch.equal(y, run(x, ids, a, b, s, base, workspace=ws))
        side = torch.cuda.Stream()
        assert torch.equal(y, run(x, ids, a, b, s, base, workspace=ws, stream=side))
        if need:
            with pytest.raises(ValueError):
                run(x, ids, a, b, s, base, stream=side)
            with pytest.raises(mg.MoeDecodeError):
                run(x, ids, a, b, s, base, workspace=ws[:256])
        out = torch.empty_like(y)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mg.moe_decode_adapters(x, ids, a, b, s, out, base=base)
        for seed in (6, 7, 8):
            x2, ids2 = make(seed, M, 256, 320, 16, 9, torch.bfloat16, dev)[:2]
            x.copy_(x2)
            ids.copy_(ids2)
            ref = run(x, ids, a, b, s, base)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, ref)


@pytest.mark.parametrize("N", [5, 9, 65, 129, 257, 1030])
def test_in_place_where_the_last_columns_are_another_wavefronts(dev, N):
    for M in (100, 2000):
        x, ids, a, b, s, base = make(N, M, 64, N, 16, 5, torch.bfloat16, dev)
        y = run(x, ids, a, b, s, base)
        mg.moe_decode_adapters(x, ids, a, b, s, base, base=base)
        assert torch.equal(base, y)


def test_refusals(dev):
    x, ids, a, b, s, base = make(9, 10, 64, 48, 16, 3, torch.bfloat16, dev)
    y = torch.empty_like(base)
    for args in ((x.half(), ids, a, b, s, y), (x.float(), ids, a, b, s, y), (x, ids.long(), a, b, s, y), (x, ids[:9], a, b, s, y),
                 (x, ids, a[:, :, :56], b, s, y), (x, ids, a, b[:, :, :8], s, y), (x, ids, a, b, s[:2], y), (x, ids, a, b, s, y[:, :40])):
        with pytest.raises(ValueError):
            mg.moe_decode_adapters(*args)
    with pytest.raises(mg.MoeDecodeError):   # R not a multiple of 8
        mg.moe_decode_adapters(x, ids, a[:, :12].contiguous(), b[:, :, :12].contiguous(), s, y)
    with pytest.raises(mg.MoeDecodeError):   # K not a multiple of 8
        mg.moe_decode_adapters(x[:, :60].contiguous(), ids, a[:, :, :60].contiguous(), b, s, y)
    wide = torch.zeros(10, 68, dtype=torch.bfloat16, device=dev)
    with pytest.raises(mg.MoeDecodeError):   # rows of x that 16-byte loads cannot take
        mg.moe_decode_adapters(wide[:, :64], ids, a, b, s, y)
    with pytest.raises(mg.MoeDecodeError):   # onto x
        mg.moe_decode_adapters(x, ids, a, b, s, x[:, :48])
    mg.moe_decode_adapters(x[:0], ids[:0], a, b, s, y[:0])
