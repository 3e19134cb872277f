"""GPU tests of moe_decode_matmul_fp8 and moe_decode_matmul_fp8_experts against
the sum of include/moe_decode.h in float64.

Tolerances.  With A = sum |x w| of an element (scales included): an FP32 y has
the rounding of its sum of K products and of the scaled blocks, (K + 2 kb + 4)
2^-24 A at the very most.  A 16-bit y may have been summed by the FP8 matrix
instruction, which cuts products off 2^-13 below the largest of their eight:
7/8 2^-10 A more at the very most, and its own rounding, eps / 2 relative (and
half of FP16's smallest step).  That worst case is far above what happens, so
the whole matrix is held to more: the error's 2-norm to the rounding's (eps / 2
of y's norm for 16 bits, 1e-6 for FP32) plus 1e-4 of y's norm for the
instruction (1.5e-5 was measured on normally distributed codes).
"""
import pytest
import torch

import moe_gate_up_amd as mg

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
VARIANTS = (0,) + tuple(getattr(mg, n) for n in sorted(dir(mg)) if n.startswith("MOE_MATMUL_"))
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def codes(g, *shape):
    """Finite E4M3 codes of normally distributed values, some of them the largest, some zero."""
    v = 60 * torch.randn(*shape, generator=g)
    u = torch.rand(*shape, generator=g)
    v = torch.where(u < 0.01, torch.full_like(v, 448.0), torch.where(u > 0.98, torch.zeros_like(v), v))
    return v.clamp(-448, 448).to(F8).view(torch.uint8)


def scales(g, *shape):
    return torch.exp(torch.randn(*shape, generator=g)) * 0.01


def values(q, s, rows):
    K = q.shape[-1]
    t = s.double().repeat_interleave(128, -1)[..., :K]
    if rows:
        t = t.repeat_interleave(128, -2)[..., : q.shape[-2], :]
    return q.view(F8).double() * t


def make(seed, M, N, K, E=0, X=None):
    g = torch.Generator().manual_seed(seed)
    X = M if X is None else X
    kb, nb = -(-K // 128), -(-N // 128)
    lead = (E,) if E else ()
    return codes(g, X, K), scales(g, X, kb), codes(g, *lead, N, K), scales(g, *lead, nb, kb)


def check(y, ref, size, K, what):
    y, eps = y.double().cpu(), torch.finfo(y.dtype).eps
    kb = -(-K // 128)
    tol = (K + 2 * kb + 4) * 2.0 ** -24 * size
    if eps > 1e-6:
        tol = tol + 7 / 8 * 2.0 ** -10 * size + eps / 2 * ref.abs() * (1 + 2.0 ** -8)
        if eps < 2.0 ** -9:
            tol = tol + 2.0 ** -25
    err = (y - ref).abs()
    assert torch.isfinite(y).all(), what
    worst = float((err / tol.clamp_min(1e-300)).max()) if y.numel() else 0.0
    rel = float((y - ref).norm() / ref.norm().clamp_min(1e-300)) if y.numel() else 0.0
    print(f"{what}: {worst:.3f} of the bound, norm {rel:.2e}", flush=True)
    assert worst <= 1, (what, worst)
    assert rel <= (1e-6 if eps < 1e-6 else eps / 2 + 1e-4), (what, rel)


def refused(out, variant):
    """The largest tile has no form for FP32 results."""
    return out == "f32" and variant == mg.MOE_MATMUL_TILE_256X256


def dense(dev, M, N, K, out, variant, seed=0, pad_x=0, pad_y=0, off_y=0):
    x, sx, w, sw = make(seed + M + N + K, M, N, K)
    X, W = values(x, sx, False), values(w, sw, True)
    ref, size = X @ W.t(), X.abs() @ W.abs().t()
    xd = torch.full((M, K + pad_x), 0x7F, dtype=torch.uint8, device=dev)   # NaN between the rows
    xd[:, :K] = x.to(dev)
    yd = torch.full((M, N + pad_y + off_y), 5.0, dtype=TYPES[out], device=dev)
    y = yd[:, off_y:off_y + N]
    if refused(out, variant):
        with pytest.raises(mg.MoeDecodeError):
            mg.moe_decode_matmul_fp8(xd[:, :K], sx.to(dev), w.to(dev), sw.to(dev), y, variant=variant)
        return
    mg.moe_decode_matmul_fp8(xd[:, :K], sx.to(dev), w.to(dev), sw.to(dev), y, variant=variant or None)
    torch.cuda.synchronize()
    check(y, ref, size, K, f"M={M} N={N} K={K} {out} variant {variant} pads {pad_x} {pad_y} {off_y}")
    assert torch.all(yd[:, off_y + N:] == 5.0) and torch.all(yd[:, :off_y] == 5.0)


SHAPES = [
    (1, 1, 16), (1, 128, 128), (1, 4096, 2048), (2, 64, 144), (5, 100, 2064), (16, 512, 4096), (17, 130, 512), (31, 257, 1040),
    (33, 96, 272), (63, 65, 64), (64, 64, 128), (65, 127, 256), (100, 300, 400), (128, 128, 1536), (129, 256, 768), (200, 1003, 1040),
    (256, 256, 128), (257, 513, 384), (300, 40, 2048), (513, 259, 640), (777, 384, 48),
    (40, 70, 8336), (130, 140, 16528), (257, 130, 24576),   # more than 64 blocks along K
]


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_one_matrix(dev, shape, variant):
    M, N, K = shape
    for out in ("bf16", "f32", "f16"):
        print(f"matmul {shape} {out} variant {variant}", flush=True)
        dense(dev, M, N, K, out, variant)


@pytest.mark.parametrize("variant", VARIANTS)
def test_strides(dev, variant):
    for M, N, K in ((3, 128, 256), (70, 132, 144), (140, 260, 528)):
        for out in ("bf16", "f32"):
            for pads in ((16, 0, 0), (48, 4, 0), (0, 3, 0), (16, 5, 1), (0, 4, 4)):
                dense(dev, M, N, K, out, variant, 9, *pads)


def test_built_in_choice_at_workload_sizes(dev):
    """Sizes of this repository's layers: one token to a prompt of 2048."""
    for M in (1, 4, 32, 100, 512, 2048):
        for N, K in ((1536, 2048), (2048, 768), (4096, 1536)):
            dense(dev, M, N, K, "bf16", 0)
    dense(dev, 300, 4096, 4096, "f32", 0)


@pytest.mark.parametrize("variant", VARIANTS)
def test_nan_and_inf_stay_in_their_rows(dev, variant):
    M, N, K = 70, 200, 400
    x, sx, w, sw = make(3, M, N, K)
    x[3, 17] = 0x7F
    sx[5, 1] = float("nan")
    w[7, 399] = 0xFF
    y = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    mg.moe_decode_matmul_fp8(x.to(dev), sx.to(dev), w.to(dev), sw.to(dev), y, variant=variant or None)
    bad = torch.isnan(y.cpu())
    want = torch.zeros(M, N, dtype=torch.bool)
    want[3] = True
    want[5] = True
    want[:, 7] = True
    assert torch.equal(bad, want)
    X, W = values(x, sx, False).nan_to_num(0), values(w, sw, True).nan_to_num(0)
    ref, size = X @ W.t(), X.abs() @ W.abs().t()
    keep = ~want
    check(y[keep.to(dev)].view(1, -1), ref[keep].view(1, -1), size[keep].view(1, -1), K, "rest")


def route(g, tokens, E, k, skew):
    s = torch.rand(tokens, E, generator=g) - skew * torch.arange(E) / E
    ids = s.topk(k, dim=1).indices.reshape(-1)
    order = torch.argsort(ids, stable=True)
    return (order // k).to(torch.int32), torch.bincount(ids, minlength=E).to(torch.int32), ids[order]


def grouped(dev, tokens, E, k, N, K, out, variant, gather=True, skew=0.0, extra=0):
    """extra: rows of y behind the last expert's, which stay as they were."""
    g = torch.Generator().manual_seed(tokens + E)
    rows, counts, expert = route(g, tokens, E, k, skew)
    M = tokens * k + extra
    x, sx, w, sw = make(tokens * k + N, tokens, N, K, E)
    X, W = values(x, sx, False)[rows.long()], values(w, sw, True)
    ref, size = torch.empty(tokens * k, N, dtype=torch.float64), torch.empty(tokens * k, N, dtype=torch.float64)
    for e in range(E):
        at = expert == e
        if at.any():
            ref[at], size[at] = X[at] @ W[e].t(), X[at].abs() @ W[e].abs().t()
    rows_d = torch.nn.functional.pad(rows, (0, extra), value=-5).to(dev)
    if gather:
        xd, sxd = x.to(dev), sx.to(dev)
    else:
        pad = torch.full((extra, K), 0x7F, dtype=torch.uint8)
        xd, sxd = torch.cat([x[rows.long()], pad]).to(dev), torch.cat([sx[rows.long()], torch.ones(extra, sx.shape[1])]).to(dev)
    y = torch.full((M, N), 5.0, dtype=TYPES[out], device=dev)
    if refused(out, variant):
        with pytest.raises(mg.MoeDecodeError):
            mg.moe_decode_matmul_fp8_experts(xd, sxd, counts.to(dev), w.to(dev), sw.to(dev), y, variant=variant,
                                             x_rows=rows_d if gather else None)
        return
    mg.moe_decode_matmul_fp8_experts(xd, sxd, counts.to(dev), w.to(dev), sw.to(dev), y, x_rows=rows_d if gather else None,
                                     variant=variant or None)
    torch.cuda.synchronize()
    check(y[: tokens * k], ref, size, K, f"experts tokens={tokens} E={E} k={k} N={N} K={K} {out} variant {variant}")
    assert torch.all(y[tokens * k:] == 5.0)


EXPERTS = [
    # tokens, E, k, N, K, skew, extra rows
    (1, 128, 8, 256, 256, 0.0, 0), (2, 3, 2, 100, 144, 0.0, 3), (32, 128, 8, 192, 512, 0.0, 0), (40, 100, 6, 130, 272, 1.0, 7),
    (100, 16, 4, 260, 384, 3.0, 70), (333, 7, 3, 129, 400, 0.5, 0), (700, 5, 2, 256, 256, 5.0, 1), (50, 1024, 8, 64, 128, 0.0, 0),
    (600, 2, 1, 300, 640, 0.0, 300), (64, 1, 1, 128, 128, 0.0, 0), (70, 65, 65, 16, 16, 0.0, 0),
]


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("shape", EXPERTS, ids=str)
def test_experts(dev, shape, variant):
    tokens, E, k, N, K, skew, extra = shape
    for out, gather in (("bf16", True), ("f32", True), ("bf16", False)):
        print(f"experts {shape} {out} gather {gather} variant {variant}", flush=True)
        grouped(dev, tokens, E, k, N, K, out, variant, gather, skew, extra)


@pytest.mark.parametrize("variant", VARIANTS)
def test_experts_odd_counts(dev, variant):
    """Empty experts, negative counts, counts beyond the rows, and row numbers outside x."""
    E, N, K, M = 9, 140, 256, 150
    x, sx, w, sw = make(5, 40, N, K, E)
    X, W = values(x, sx, False), values(w, sw, True)
    g = torch.Generator().manual_seed(4)
    rows = torch.randint(0, 40, (M,), generator=g, dtype=torch.int32)
    rows[10], rows[77], rows[120] = -1, 40, 2 ** 31 - 1
    for counts, ends in (([0] * 9, []), ([-3, 20, 0, 70, -2147483648, 1, 0, 30, 0], [0, 20, 20, 90, 90, 91, 91, 121, 121]),
                         ([100, 0, 2147483647, 5, 5, 5, 5, 5, 5], [100, 100, 150]), ([0] * 8 + [1], [0] * 8 + [1])):
        out = torch.bfloat16 if refused("f32", variant) else torch.float32
        y = torch.full((M, N), 5.0, dtype=out, device=dev)
        mg.moe_decode_matmul_fp8_experts(x.to(dev), sx.to(dev), torch.tensor(counts, dtype=torch.int32, device=dev), w.to(dev),
                                         sw.to(dev), y, x_rows=rows.to(dev), variant=variant or None)
        torch.cuda.synchronize()
        done, y = 0, y.cpu()
        for e, end in enumerate(ends):
            for m in range(done, end):
                r = int(rows[m])
                if 0 <= r < 40:
                    ref, size = X[r] @ W[e].t(), X[r].abs() @ W[e].abs().t()
                    tol = (K + 8) * 2.0 ** -24 * size + 1e-30
                    if out == torch.bfloat16:
                        tol = tol + 7 / 8 * 2.0 ** -10 * size + 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -8)
                    assert torch.all((y[m].double() - ref).abs() <= tol), (counts, m)
                else:
                    assert torch.isnan(y[m]).all(), (counts, m)
            done = end
        assert torch.all(y[done:] == 5.0), counts


def test_same_bits_and_capture(dev):
    E, k, N, K, tokens = 16, 4, 320, 512, 90
    g = torch.Generator().manual_seed(1)
    rows, counts, _ = route(g, tokens, E, k, 0.5)
    x, sx, w, sw = (t.to(dev) for t in make(2, tokens, N, K, E))
    rows, counts = rows.to(dev), counts.to(dev)
    y = torch.empty(tokens * k, N, dtype=torch.bfloat16, device=dev)
    call = lambda: mg.moe_decode_matmul_fp8_experts(x, sx, counts, w, sw, y, x_rows=rows)   # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for rep in range(3):
        r2, c2, _ = route(g, tokens, E, k, rep)
        rows.copy_(r2)
        counts.copy_(c2)
        call()
        torch.cuda.synchronize()
        eager = y.clone()
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager), rep
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y2 = torch.empty_like(y)
    mg.moe_decode_matmul_fp8_experts(x, sx, counts, w, sw, y2, x_rows=rows, stream=st)
    st.synchronize()
    assert torch.equal(y2, eager)


def test_rows_beyond_32_bit_offsets(dev):
    """x and y whose rows lie beyond 2^32 bytes from their start."""
    M, N, K, ld = 9, 256, 256, 1 << 29
    x, sx, w, sw = make(8, M, N, K)
    xd = torch.empty((M - 1) * ld + K, dtype=torch.uint8, device=dev).as_strided((M, K), (ld, 1))
    xd.copy_(x.to(dev))
    yd = torch.empty((M - 1) * ld + N, dtype=torch.bfloat16, device=dev).as_strided((M, N), (ld, 1))
    X, W = values(x, sx, False), values(w, sw, True)
    for variant in VARIANTS:
        yd.zero_()
        try:
            mg.moe_decode_matmul_fp8(xd, sx.to(dev), w.to(dev), sw.to(dev), yd, variant=variant or None)
        except mg.MoeDecodeError as e:   # a variant whose 32-bit offsets do not reach a tile's rows refuses the call
            assert variant and e.code == mg.MOE_ERR_ARG
            continue
        torch.cuda.synchronize()
        check(yd.contiguous(), X @ W.t(), X.abs() @ W.abs().t(), K, f"far rows variant {variant}")


def test_experts_rows_beyond_32_bit_offsets(dev):
    """Rows picked from a tensor of more than 2^32 bytes."""
    tokens, E, k, N, K, ld = 9, 3, 2, 200, 272, 1 << 29
    g = torch.Generator().manual_seed(3)
    rows, counts, expert = route(g, tokens, E, k, 0.0)
    x, sx, w, sw = make(8, tokens, N, K, E)
    xd = torch.empty((tokens - 1) * ld + K, dtype=torch.uint8, device=dev).as_strided((tokens, K), (ld, 1))
    xd.copy_(x.to(dev))
    X, W = values(x, sx, False)[rows.long()], values(w, sw, True)
    ref = torch.stack([X[m] @ W[expert[m]].t() for m in range(tokens * k)])
    size = torch.stack([X[m].abs() @ W[expert[m]].abs().t() for m in range(tokens * k)])
    for variant in (0, mg.MOE_MATMUL_ROWS_16, mg.MOE_MATMUL_FAR_ROWS):
        y = torch.empty(tokens * k, N, dtype=torch.float32, device=dev)
        mg.moe_decode_matmul_fp8_experts(xd, sx.to(dev), counts.to(dev), w.to(dev), sw.to(dev), y, x_rows=rows.to(dev),
                                         variant=variant or None)
        torch.cuda.synchronize()
        check(y, ref, size, K, f"far picked rows variant {variant}")


def test_experts_matrices_beyond_4_gib(dev):
    """The last of 200 experts' matrices lies beyond 2^32 bytes."""
    E, N, K = 200, 4096, 8192
    g = torch.Generator().manual_seed(6)
    w = torch.zeros(E, N, K, dtype=torch.uint8, device=dev)
    sw = torch.ones(E, N // 128, K // 128, device=dev)
    last, s_last = codes(g, N, K), scales(g, N // 128, K // 128)
    w[-1] = last.to(dev)
    sw[-1] = s_last.to(dev)
    x, sx = codes(g, 20, K), scales(g, 20, K // 128)
    counts = torch.zeros(E, dtype=torch.int32, device=dev)
    counts[0], counts[-1] = 4, 16
    X, W = values(x, sx, False), values(last, s_last, True)
    for variant in VARIANTS:
        y = torch.empty(20, N, dtype=torch.bfloat16, device=dev)
        mg.moe_decode_matmul_fp8_experts(x.to(dev), sx.to(dev), counts, w, sw, y, variant=variant or None)
        torch.cuda.synchronize()
        assert torch.count_nonzero(y[:4]) == 0
        check(y[4:], X[4:] @ W.t(), X[4:].abs() @ W.abs().t(), K, f"last expert variant {variant}")


def test_refusals(dev):
    z = lambda *s, dtype=torch.uint8: torch.zeros(*s, dtype=dtype, device=dev)   # noqa: E731
    f = torch.float32
    x, sx, w, sw, y = z(4, 256), z(4, 2, dtype=f), z(128, 256), z(1, 2, dtype=f), z(4, 128, dtype=torch.bfloat16)
    for bad in ((x.float(), sx, w, sw, y), (x, sx[:3], w, sw, y), (x, sx, w[:, :128], sw, y), (x, sx, w, sw.double(), y),
                (x, sx, w, sw, y[:3]), (x, sx, w, sw, y.double()), (x, sx, w, sw, z(128, 4, dtype=torch.bfloat16).t()),
                (z(256, 4).t(), sx, w, sw, y), (x, sx, w.t(), sw, y)):
        with pytest.raises(ValueError):
            mg.moe_decode_matmul_fp8(*bad)
    with pytest.raises(mg.MoeDecodeError):   # K not a multiple of 16
        mg.moe_decode_matmul_fp8(z(4, 40), z(4, 1, dtype=f), z(8, 40), z(1, 1, dtype=f), z(4, 8, dtype=f))
    we, swe, c = z(3, 128, 256), z(3, 1, 2, dtype=f), z(3, dtype=torch.int32)
    for bad in ((x, sx, c[:2], we, swe, y), (x, sx, c.long(), we, swe, y), (x, sx, c, we, swe[:2], y)):
        with pytest.raises(ValueError):
            mg.moe_decode_matmul_fp8_experts(*bad)
    with pytest.raises(ValueError):
        mg.moe_decode_matmul_fp8_experts(x, sx, c, we, swe, y, x_rows=z(3, dtype=torch.int32))
    with pytest.raises(mg.MoeDecodeError):   # more rows of y than of x, and no row numbers
        mg.moe_decode_matmul_fp8_experts(x, sx, c, we, swe, z(5, 128, dtype=f))
    mg.moe_decode_matmul_fp8(x[:0], sx[:0], w, sw, y[:0])


def test_two_calls_at_once(dev):
    """A product of one matrix and an experts' one on streams of their own, reading the same rows: the bits of each alone."""
    E, k, N, K, tokens = 16, 4, 384, 1024, 300
    g = torch.Generator().manual_seed(8)
    rows, counts, _ = route(g, tokens, E, k, 0.3)
    x, sx, w, sw = (t.to(dev) for t in make(9, tokens, N, K, E))
    rows, counts = rows.to(dev), counts.to(dev)
    y = [torch.empty(tokens, N, dtype=torch.bfloat16, device=dev), torch.empty(tokens * k, N, dtype=torch.bfloat16, device=dev)]
    one = lambda out, st: mg.moe_decode_matmul_fp8(x, sx, w[3], sw[3], out, stream=st)   # noqa: E731
    many = lambda out, st: mg.moe_decode_matmul_fp8_experts(x, sx, counts, w, sw, out, x_rows=rows, stream=st)   # noqa: E731
    one(y[0], None)
    many(y[1], None)
    torch.cuda.synchronize()
    alone = [t.clone() for t in y]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for t in y:
            t.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            one(y[0], streams[0])
            many(y[1], streams[1])
        torch.cuda.synchronize()
        assert torch.equal(y[0], alone[0]) and torch.equal(y[1], alone[1])


def test_overlapping_rows_of_one_tensor(dev):
    """x and the rows of y as columns of one larger tensor each, with sizes that end inside every tile."""
    M, N, K = 131, 200, 272
    x, sx, w, sw = make(21, M, N, K)
    X, W = values(x, sx, False), values(w, sw, True)
    big = torch.full((M, 3 * K), 0x7F, dtype=torch.uint8, device=dev)
    big[:, K:2 * K] = x.to(dev)
    out = torch.full((M, 3 * N), 5.0, dtype=torch.float16, device=dev)
    mg.moe_decode_matmul_fp8(big[:, K:2 * K], sx.to(dev), w.to(dev), sw.to(dev), out[:, N:2 * N])
    torch.cuda.synchronize()
    check(out[:, N:2 * N], X @ W.t(), X.abs() @ W.abs().t(), K, "columns of a larger tensor")
    assert torch.all(out[:, :N] == 5.0) and torch.all(out[:, 2 * N:] == 5.0)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("counts", [[17] * 41, [256] * 8, [261, 3, 0, 512, 64, 65, 33, 127, 128, 129, 32, 1] * 2, [1] * 300, [700]],
                         ids=["all short", "all whole", "both", "single rows", "one"])
def test_experts_whole_and_short_tiles(dev, counts, variant):
    """Every tile of y is computed once, whatever share of them is whole and whatever the XCDs' shares come to."""
    E, N, K, M = len(counts), 330, 144, sum(counts)
    x, sx, w, sw = make(E + M, M, N, K, E)
    X, W = values(x, sx, False), values(w, sw, True)
    ref, size = torch.empty(M, N, dtype=torch.float64), torch.empty(M, N, dtype=torch.float64)
    first = 0
    for e, c in enumerate(counts):
        rows = slice(first, first + c)
        ref[rows], size[rows] = X[rows] @ W[e].t(), X[rows].abs() @ W[e].abs().t()
        first += c
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=dev)
    mg.moe_decode_matmul_fp8_experts(x.to(dev), sx.to(dev), torch.tensor(counts, dtype=torch.int32, device=dev), w.to(dev),
                                     sw.to(dev), y, variant=variant or None)
    torch.cuda.synchronize()
    check(y, ref, size, K, f"{E} experts, {M} rows, variant {variant}")
