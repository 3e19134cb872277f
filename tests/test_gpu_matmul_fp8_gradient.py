"""GPU tests of the products' gradient with respect to x, made with the same calls: dy quantised in blocks of 128 along
N, times w^T with sw^T.

Against the formula dx = dy w in float64 on the quantised dy, to the bounds of FP32 sums over N ((N + 2 nb + 4) 2^-24 of the
sum of magnitudes and the result's rounding), and against differences: y is linear in x, so the central difference of
L = sum(dy y) along any direction v is sum(dx v) whatever the step, and the product's dx is off by the same bounds times |v|.
"""
import pytest
import torch

import moe_gate_up_amd as mg
from tests.test_gpu_matmul_fp8 import TYPES, codes, route, scales, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def quantised(dy, dev):
    M, N = dy.shape
    q, s = torch.empty(M, N, dtype=torch.uint8, device=dev), torch.empty(M, -(-N // 128), device=dev)
    mg.moe_decode_quantize_fp8(dy.to(dev), q, s)
    return q, s


def bound(size, ref, N, out):
    tol = (N + 2 * -(-N // 128) + 4) * 2.0 ** -24 * size
    if out != "f32":
        tol = tol + torch.finfo(TYPES[out]).eps / 2 * (1 + 2.0 ** -8) * ref.abs()
    return tol + (2.0 ** -25 if out == "f16" else 0)


def differences(loss, x, dx, tol, g):
    for _ in range(3):
        v = torch.randn(x.shape, generator=g, dtype=torch.float64)
        num = float((loss(x + v) - loss(x - v)) / 2)
        got = float((dx * v).sum())
        assert abs(num - got) <= float((tol * v.abs()).sum()) + 1e-12 * abs(num), (num, got)


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(1, 128, 256), (5, 80, 400), (70, 272, 144), (300, 1040, 528)], ids=str)
def test_one_matrix(dev, shape, out):
    M, N, K = shape
    print(f"gradient {shape} {out}", flush=True)
    g = torch.Generator().manual_seed(M)
    w, sw = codes(g, N, K), scales(g, -(-N // 128), -(-K // 128))
    q, s = quantised(torch.randn(M, N, generator=g), dev)
    dx = torch.empty(M, K, dtype=TYPES[out], device=dev)
    mg.moe_decode_matmul_fp8(q, s, w.t().contiguous().to(dev), sw.t().contiguous().to(dev), dx)
    DY, W = values(q.cpu(), s.cpu(), False), values(w, sw, True)
    ref = DY @ W
    tol = bound(DY.abs() @ W.abs(), ref, N, out)
    dx = dx.cpu().double()
    assert bool(((dx - ref).abs() <= tol).all())
    differences(lambda x: (DY * (x @ W.t())).sum(), torch.randn(M, K, generator=g, dtype=torch.float64), dx, tol, g)


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_experts(dev, out):
    """Every token stands in k rows: its gradient is their sum."""
    tokens, E, k, N, K = 90, 7, 3, 208, 272
    print(f"gradient through experts {out}", flush=True)
    g = torch.Generator().manual_seed(5)
    rows, counts, expert = route(g, tokens, E, k, 1.0)
    w, sw = codes(g, E, N, K), scales(g, E, 2, 3)
    q, s = quantised(torch.randn(tokens * k, N, generator=g), dev)
    part = torch.empty(tokens * k, K, dtype=TYPES[out], device=dev)
    mg.moe_decode_matmul_fp8_experts(q, s, counts.to(dev), w.transpose(1, 2).contiguous().to(dev),
                                     sw.transpose(1, 2).contiguous().to(dev), part)
    DY, W = values(q.cpu(), s.cpu(), False), values(w, sw, True)
    ref = torch.stack([DY[m] @ W[expert[m]] for m in range(tokens * k)])
    tol = bound(torch.stack([DY[m].abs() @ W[expert[m]].abs() for m in range(tokens * k)]), ref, N, out)
    part = part.cpu().double()
    assert bool(((part - ref).abs() <= tol).all())
    summed = lambda t: torch.zeros(tokens, K, dtype=torch.float64).index_add_(0, rows.long(), t)   # noqa: E731
    x = torch.randn(tokens, K, generator=g, dtype=torch.float64)
    loss = lambda t: sum((DY[m] * (W[expert[m]] @ t[rows[m]])).sum() for m in range(tokens * k))   # noqa: E731
    differences(loss, x, summed(part), summed(tol), g)
