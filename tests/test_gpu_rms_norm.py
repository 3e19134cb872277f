"""GPU tests of moe_decode_rms_norm and its gradients against the definition in
include/moe_decode.h, in float64 on the CPU.

Tolerances, u = 2^-24.  The stored sum is one FP32 addition and one rounding: exact.  The
squares are a chain of at most 64 fused multiply-adds in a lane, 6 steps over the lanes and
16 over wavefronts: 86 u of a sum of positive terms, the root halves that, and mean, eps,
root and quotient cost 4 u: rstd within 50 u, v = r rstd w within 52 u.  A code stands
for v within half a step (2^-4 relative, 2^-10 scales below E4M3's normal numbers), its scale
within 54 u.
Gradients, given rstd as it was stored: n = r rstd within u, the mean of dy w n within
90 u of its terms' magnitudes, dx within rstd (4 u |dy w| + |n| 96 u mean |dy w n|), 2 u
of the sum with dsum, and one rounding.  dweight: a chain of at most M / 512 + 8 additions in
FP32 (FP64 behind), each term within 2 u.
"""
import pytest
import torch

import moe_gate_up_amd as mg

pytestmark = pytest.mark.gpu
U, TINY = 2.0 ** -24, 1.2e-38
TYPES = [torch.bfloat16, torch.float16, torch.float32]
EPS = 1e-6
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def half(dtype):
    return torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0.0


def small(dtype):
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def make(seed, M, H, dtype, wtype, dev):
    g = torch.Generator().manual_seed(seed)
    gain = torch.exp(0.5 * torch.randn(H, generator=g)) * (1 + 20 * (torch.rand(H, generator=g) < 0.01))
    x, res = ((torch.randn(M, H, generator=g) * gain).to(dtype).to(dev) for _ in range(2))
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(wtype).to(dev)
    return x, res, w


def forward(x, res, w, q=True, pow2=False, eps=EPS, y=None):
    M, H = x.shape
    y = torch.full((M, H), 7.0, dtype=x.dtype, device=x.device) if y is None else y
    total = None if res is None else torch.full((M, H), 7.0, dtype=x.dtype, device=x.device)
    codes = torch.full((M, H), 0xAA, dtype=torch.uint8, device=x.device) if q else None
    s = torch.full((M, -(-H // 128)), -1.0, device=x.device) if q else None
    rstd = torch.full((M,), -1.0, device=x.device)
    mg.moe_decode_rms_norm(x, w, eps, y=y, q=codes, scales=s, residual=res, sum_out=total, rstd=rstd, pow2=pow2)
    torch.cuda.synchronize()
    return y, total, codes, s, rstd


def values(x, res, w, eps=EPS):
    r = x.cpu() if res is None else (x.cpu().float() + res.cpu().float()).to(x.dtype)
    d = r.double()
    rstd = 1 / torch.sqrt(d.square().mean(1) + eps)
    return r, rstd, d * rstd[:, None] * w.cpu().double()


def check_codes(codes, s, v, pow2):
    M, H = v.shape
    pad = torch.nn.functional.pad(v, (0, -H % 128)).view(M, -1, 128)
    rs = (pad.abs().amax(-1) / 448).clamp_min(2.0 ** -126)
    s = s.cpu().double()
    if pow2:
        assert bool((torch.frexp(s).mantissa == 0.5).all())
        assert bool((s >= rs * (1 - 60 * U)).all()) and bool((s <= 2 * rs * (1 + 60 * U)).all())
    else:
        assert bool(((s - rs).abs() <= 54 * U * rs + TINY).all())
    wide = s.repeat_interleave(128, 1)[:, :H]
    got = codes.cpu().view(F8).double() * wide
    assert bool(((got - v).abs() <= 2.0 ** -4 * v.abs() * (1 + 60 * U) + 2.0 ** -10 * wide + 60 * U * v.abs()).all())


def check(x, res, w, pow2=False):
    y, total, codes, s, rstd = forward(x, res, w, pow2=pow2)
    r, rr, v = values(x, res, w)
    if res is not None:
        assert torch.equal(total.cpu(), r)
    assert bool(((rstd.cpu().double() - rr).abs() <= 50 * U * rr).all())
    assert bool(((y.cpu().double() - v).abs() <= 52 * U * v.abs() + half(x.dtype) * v.abs() * (1 + 52 * U) + small(x.dtype)).all())
    check_codes(codes, s, v, pow2)
    only, _, _, _, _ = forward(x, res, w, q=False)
    assert torch.equal(only, y)


SHAPES = [(1, 1), (3, 7), (5, 8), (2, 127), (4, 128), (9, 129), (33, 512), (3, 513), (777, 1003), (32, 2048), (2, 2049), (37, 4096),
          (3, 4100), (5, 8192), (2, 10000), (3, 16384), (2, 16385), (2, 32768)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(dev, shape, dtype):
    M, H = shape
    print(f"norm {shape} {dtype}", flush=True)
    for wtype in {dtype, torch.float32}:
        x, res, w = make(M + H, M, H, dtype, wtype, dev)
        check(x, res, w)
        check(x, None, w, pow2=True)


def backward(dy, r, w, rstd, dsum, **kw):
    dx = torch.full_like(r, 7.0)
    dw = torch.full((r.shape[1],), 7.0, device=r.device)
    mg.moe_decode_rms_norm_backward(dy, r, w, rstd, dx, dw, dsum=dsum, **kw)
    torch.cuda.synchronize()
    return dx, dw


def check_backward(dy, r, w, rstd, dsum):
    M, H = r.shape
    dx, dw = backward(dy, r, w, rstd, dsum)
    g, n = dy.cpu().double(), r.cpu().double() * rstd.cpu().double()[:, None]
    gw, rs = g * w.cpu().double(), rstd.cpu().double()[:, None]
    ref = rs * (gw - n * (gw * n).mean(1, keepdim=True))
    err = rs * (4 * U * gw.abs() + n.abs() * 96 * U * (gw * n).abs().mean(1, keepdim=True))
    if dsum is not None:
        ref = ref + dsum.cpu().double()
        err = err + 2 * U * (ref.abs() + dsum.cpu().double().abs())
    assert bool(((dx.cpu().double() - ref).abs() <= err + half(r.dtype) * (ref.abs() + err) + small(r.dtype)).all())
    rw, size = (g * n).sum(0), (g * n).abs().sum(0)
    assert bool(((dw.cpu().double() - rw).abs() <= (M / 512 + 8) * U * size + TINY).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES + [(3001, 256), (2500, 2000), (600, 5000), (9000, 40)], ids=str)
def test_backward(dev, shape, dtype):
    M, H = shape
    print(f"norm backward {shape} {dtype}", flush=True)
    for wtype in {dtype, torch.float32}:
        x, res, w = make(M + H, M, H, dtype, wtype, dev)
        _, r, _, _, rstd = forward(x, res, w, q=False)
        g = torch.Generator().manual_seed(M)
        dy, dsum = (torch.randn(M, H, generator=g).to(dtype).to(dev) for _ in range(2))
        check_backward(dy, r, w, rstd, dsum)
        check_backward(dy, r, w, rstd, None)


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_alignment_and_in_place(dev, dtype):
    M, H = 10, 264
    x, res, w = make(1, M, H, dtype, dtype, dev)
    y, total, codes, s, rstd = forward(x, res, w)
    dy = torch.randn(M, H, generator=torch.Generator().manual_seed(2)).to(dtype).to(dev)
    dx, dw = backward(dy, total, w, rstd, res)
    for pad, off in ((8, 0), (3, 1), (0, 5)):
        def wide(t):
            b = torch.full((M, H + pad + off), 2.0, dtype=dtype, device=dev)
            b[:, off:off + H] = t
            return b, b[:, off:off + H]
        (_, x2), (rb, r2), (yb, y2) = wide(x), wide(res), wide(torch.zeros_like(y))
        w2 = torch.cat([w[:1], w])[1:]
        c2, s2, d2 = torch.empty_like(codes), torch.empty_like(s), torch.empty_like(rstd)
        mg.moe_decode_rms_norm(x2, w2, EPS, y=y2, q=c2, scales=s2, residual=r2, sum_out=r2, rstd=d2)   # the sum onto the residual
        assert torch.equal(y2, y) and torch.equal(r2, total) and torch.equal(c2, codes) and torch.equal(s2, s) and torch.equal(d2, rstd)
        (_, g2), (sb, s3) = wide(dy), wide(res)
        dw2 = torch.empty_like(dw)
        mg.moe_decode_rms_norm_backward(g2, r2, w2, d2, s3, dw2, dsum=s3)   # onto the gradient that is added
        assert torch.equal(s3, dx) and torch.equal(dw2, dw)
        for b in (rb, yb, sb):
            b[:, off:off + H] = 2.0
            assert bool((b == 2.0).all())
    q2, s2 = torch.empty_like(codes), torch.empty_like(s)
    mg.moe_decode_rms_norm(x, w, EPS, q=q2, scales=s2, residual=res)   # 8 bits alone
    assert torch.equal(q2, codes) and torch.equal(s2, s)


def test_zero_large_and_not_finite_rows(dev):
    H = 640
    for dtype in (torch.bfloat16, torch.float32):
        x, _, w = make(3, 12, H, dtype, dtype, dev)
        x[0] = 0
        x[1] = 3e38 * torch.sign(x[1])       # squares pass FP32
        x[2] *= 1e20
        x[3] *= 1e-25
        x[4, 7] = float("nan")
        x[5, 9] = float("inf")
        x[6] = 0
        x[6, 3] = 3e38
        y, _, codes, s, rstd = forward(x, None, w)
        _, rr, v = values(x, None, w)
        on = [0, 1, 2, 3, 6, 7, 8, 9, 10, 11]
        # a subnormal rstd (row 1) is off by up to 2^-150
        rel = 52 * U + (2.0 ** -150 / rr)
        assert bool(((rstd.cpu().double() - rr).abs() <= rel * rr)[on].all())
        assert bool(((y.cpu().double() - v).abs() <= (rel[:, None] + half(dtype) * 1.01) * v.abs() + small(dtype))[on].all())
        assert bool(torch.isnan(y[4]).all())
        assert bool(torch.isnan(y[5, 9])) and bool((y[5, :9] == 0).all()) and bool((y[5, 10:] == 0).all())
        assert bool((codes[4] == 0x7F).all()) and int(codes[5, 9]) == 0x7F
        assert bool((y[0] == 0).all()) and bool(torch.isfinite(y[on].float()).all())


def test_gradient_against_differences(dev):
    """Of the definition in float64: (f(x + h) - f(x - h)) / 2h, whose own error is h^2 and 1e-16 / h."""
    M, H, h = 3, 20, 1e-5
    x, _, w = make(4, M, H, torch.float32, torch.float32, dev)
    dy = torch.randn(M, H, generator=torch.Generator().manual_seed(5)).to(dev)
    _, _, _, _, rstd = forward(x, None, w, q=False)
    dx, dw = backward(dy, x, w, rstd, None)

    def value(xx, ww):
        return (xx / torch.sqrt(xx.square().mean(1, keepdim=True) + EPS) * ww * dy.cpu().double()).sum(1)
    xd, wd = x.cpu().double(), w.cpu().double()
    for c in range(H):
        step = torch.zeros(M, H, dtype=torch.float64)
        step[:, c] = h
        diff = (value(xd + step, wd) - value(xd - step, wd)) / (2 * h)
        assert bool(((dx[:, c].cpu().double() - diff).abs() <= 2e-5 * (1 + diff.abs())).all())
        dwc = float((value(xd, wd + step[0]) - value(xd, wd - step[0])).sum()) / (2 * h)
        assert abs(float(dw[c]) - dwc) <= 2e-5 * (1 + abs(dwc))


def test_graph_stream_and_repeat(dev):
    M, H = 1500, 1024
    x, res, w = make(6, M, H, torch.bfloat16, torch.bfloat16, dev)
    dy = torch.randn(M, H, generator=torch.Generator().manual_seed(7)).to(torch.bfloat16).to(dev)
    ws = torch.full((mg.moe_decode_rms_norm_backward_workspace(M, H),), 0xAB, dtype=torch.uint8, device=dev)
    y, total, codes, s, rstd = forward(x, res, w)
    dx, dw = backward(dy, total, w, rstd, res, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip((dx, dw), backward(dy, total, w, rstd, res)))
    side = torch.cuda.Stream()
    assert all(torch.equal(a, b) for a, b in zip((dx, dw), backward(dy, total, w, rstd, res, workspace=ws, stream=side)))
    with pytest.raises(ValueError):
        backward(dy, total, w, rstd, res, stream=side)
    outs = [torch.empty_like(t) for t in (y, total, codes, s, rstd, dx, dw)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mg.moe_decode_rms_norm(x, w, EPS, y=outs[0], q=outs[2], scales=outs[3], residual=res, sum_out=outs[1], rstd=outs[4])
        mg.moe_decode_rms_norm_backward(dy, outs[1], w, outs[4], outs[5], outs[6], dsum=res)
    for seed in (1, 2, 3):
        x.copy_(make(seed, M, H, torch.bfloat16, torch.bfloat16, dev)[0])
        ref = forward(x, res, w)
        ref += backward(dy, ref[1], w, ref[4], res)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))


@pytest.mark.parametrize("H", [5, 9, 513, 1025, 1031, 1537, 2049, 4097, 6145, 8193, 16385])
def test_in_place_where_the_last_columns_are_another_wavefronts(dev, H):
    """The last columns, fewer than 8, begin where a wavefront's share ends: the sum onto the residual and dx onto dsum
    are as out of place."""
    for dtype in (torch.bfloat16, torch.float32):
        M = 600
        x, res, w = make(H, M, H, dtype, dtype, dev)
        y, total, _, _, rstd = forward(x, res, w, q=False)
        dy = torch.randn(M, H, generator=torch.Generator().manual_seed(H)).to(dtype).to(dev)
        dx, dw = backward(dy, total, w, rstd, res)
        r2, y2, s2, dw2 = res.clone(), torch.empty_like(y), res.clone(), torch.empty_like(dw)
        mg.moe_decode_rms_norm(x, w, EPS, y=y2, residual=r2, sum_out=r2)
        mg.moe_decode_rms_norm_backward(dy, total, w, rstd, s2, dw2, dsum=s2)
        assert torch.equal(r2, total) and torch.equal(y2, y) and torch.equal(s2, dx) and torch.equal(dw2, dw)


def test_refusals(dev):
    x, res, w = make(8, 6, 64, torch.bfloat16, torch.bfloat16, dev)
    y, q, s = torch.empty_like(x), torch.empty(6, 64, dtype=torch.uint8, device=dev), torch.empty(6, 1, device=dev)
    for kw in (dict(y=y.float()), dict(y=y[:5]), dict(y=y, residual=res.half()), dict(q=q[:, :63], scales=s), dict(q=q, scales=s.view(6)), dict(y=y.t())):
        with pytest.raises(ValueError):
            mg.moe_decode_rms_norm(x, w, EPS, **kw)
    for kw in (dict(), dict(q=q), dict(scales=s, y=y), dict(y=y, sum_out=torch.empty_like(x)), dict(y=x), dict(y=y, residual=res, sum_out=x),
               dict(y=res, residual=res)):
        with pytest.raises(mg.MoeDecodeError):
            mg.moe_decode_rms_norm(x, w, EPS, **kw)
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(mg.MoeDecodeError):
            mg.moe_decode_rms_norm(x, w, eps, y=y)
    with pytest.raises(ValueError):
        mg.moe_decode_rms_norm(x, w.half(), EPS, y=y)
    with pytest.raises(mg.MoeDecodeError):
        mg.moe_decode_rms_norm(torch.empty(1, 32769, device=dev), torch.ones(32769, device=dev), EPS, y=torch.empty(1, 32769, device=dev))
    rstd, dw = torch.ones(6, device=dev), torch.empty(64, device=dev)
    with pytest.raises(mg.MoeDecodeError):
        mg.moe_decode_rms_norm_backward(y, x, w, rstd, x, dw)
    with pytest.raises(mg.MoeDecodeError):
        mg.moe_decode_rms_norm_backward(y, x, w, rstd, res, dw, workspace=torch.empty(256, dtype=torch.uint8, device=dev))
    mg.moe_decode_rms_norm(x[:0], w, EPS, y=y[:0])
    dw.fill_(3.0)
    mg.moe_decode_rms_norm_backward(y[:0], x[:0], w, rstd[:0], res[:0], dw)
    torch.cuda.synchronize()
    assert bool((dw == 3.0).all())
