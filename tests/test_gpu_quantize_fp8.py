"""GPU tests of moe_decode_quantize_fp8 against its definition in
include/moe_decode.h.

Without SwiGLU both divisions are FP32 divisions rounded correctly and the
conversion is to nearest even, so scales and codes equal the host's bit for
bit (PyTorch on the CPU; float32 division there is correctly rounded).

With SwiGLU v = silu(g) u is computed in FP32: exp(-g) costs |g| 2^-24 / ln 2
relative, the sum, the quotient and the product a few 2^-24 more, so v is
within (|g| + 4) 2^-23 relative of the exact value.  A scale is then within
that of the largest value's, and a code's value within half a step of v
(2^-4 relative, or 2^-10 scales below E4M3's normal numbers) plus v's error.
"""
import numpy as np
import pytest
import torch

import moe_gate_up_amd as mg

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def blocks(v):
    K = v.shape[1]
    return torch.nn.functional.pad(v, (0, -K % 128)).view(v.shape[0], -1, 128)


def reference(x, pow2=False):
    """Scales and codes of float32 x on the CPU."""
    v = blocks(x)
    a = torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v)).amax(-1)
    s = torch.maximum(a / torch.tensor(448.0), torch.tensor(2.0 ** -126))
    if pow2:
        b = s.numpy().view(np.uint32)
        s = torch.from_numpy((((b + 0x7FFFFF) >> 23) << 23).astype(np.uint32).view(np.float32).copy())
    q = (v / s[..., None]).to(F8).view(torch.uint8)
    q = torch.where(torch.isfinite(v), q, torch.full_like(q, 0x7F))
    return q.reshape(x.shape[0], -1)[:, :x.shape[1]], s


def run(x, K, swiglu=False, pow2=False):
    M = x.shape[0]
    q = torch.full((M, K), 0xAA, dtype=torch.uint8, device=x.device)
    s = torch.full((M, -(-K // 128)), -1.0, device=x.device)
    mg.moe_decode_quantize_fp8(x, q, s, swiglu=swiglu, pow2=pow2)
    torch.cuda.synchronize()
    return q.cpu(), s.cpu()


def same(got, ref, what):
    (q, s), (rq, rs) = got, ref
    assert torch.equal(s.view(torch.int32), rs.view(torch.int32)), (what, (s != rs).nonzero()[:4])
    bad = (q != rq).nonzero()
    assert bad.numel() == 0, (what, bad[:4], q[tuple(bad[0])].item(), rq[tuple(bad[0])].item())


SHAPES = [(1, 1), (1, 16), (1, 128), (3, 127), (5, 129), (2, 8), (7, 136), (33, 768), (4, 2048), (1000, 72), (2, 4095), (300, 4096), (1, 8192)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_bit_exact(dev, shape, dtype):
    M, K = shape
    print(f"quantize {shape} {dtype}", flush=True)
    g = torch.Generator().manual_seed(M * K)
    x = (torch.randn(M, K, generator=g) * torch.exp(2 * torch.randn(M, 1, generator=g))).to(dtype)
    for pow2 in (False, True):
        same(run(x.to(dev), K, pow2=pow2), reference(x.float(), pow2), (shape, dtype, pow2))
    # rows apart, and a start that 16-byte loads cannot take
    for pad, off in ((8, 0), (3, 0), (8, 1)):
        wide = torch.randn(M, K + pad + off).to(dtype)
        wide[:, off:off + K] = x
        same(run(wide.to(dev)[:, off:off + K], K), reference(x.float()), (shape, dtype, "strided", pad, off))


def test_special_values(dev):
    """Zeros, signed zeros, subnormal and tiny blocks, the largest values, NaN and infinities, ties."""
    K = 128 * 12
    x = torch.randn(4, K, generator=torch.Generator().manual_seed(0))
    x[0, 0:128] = 0
    x[0, 1] = -0.0
    x[0, 128:256] = 1e-40
    x[0, 256:384] *= 1e-38
    x[0, 384:512] *= 1e-30
    x[0, 512:640] = 3.4e38
    x[0, 640:768] *= 1e38
    x[0, 700] = float("nan")
    x[0, 768] = float("inf")
    x[0, 769] = -float("inf")
    x[0, 896:1024] = float("nan")
    x[0, 1024:1152] = float("-inf")
    x[0, 1152:1280] = torch.arange(128) * 3.5      # amax 444.5
    x[0, 1280:1408] = torch.arange(128) / 16 * 448 / 7.9375
    x[0, 1408:1536] = 1.4013e-45
    x[1] = torch.linspace(-448, 448, K)
    x[2] = torch.linspace(-1e-36, 1e-36, K)
    x[3] = torch.linspace(-3e-33, 1e-33, K)
    for pow2 in (False, True):
        same(run(x.to(dev), K, pow2=pow2), reference(x, pow2), ("special", pow2))
    h = x.clone()
    h[:, ::7] = 60000.0
    hh = h.half()
    same(run(hh.to(dev), K), reference(hh.float()), "half")
    b = x.to(torch.bfloat16)
    same(run(b.to(dev), K), reference(b.float()), "bfloat16")


def test_every_bf16_value(dev):
    """All 65536 bf16 patterns, in blocks of neighbours and in blocks that span the range."""
    v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    for x in (v.view(512, 128), v.view(128, 512).t().contiguous().view(128, 512)):
        same(run(x.contiguous().to(dev), x.shape[1]), reference(x.float()), "every bf16")
        same(run(x.view(torch.int16).contiguous().to(dev), x.shape[1]), reference(x.float()), "as patterns")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 128), (3, 127), (5, 136), (65, 768), (2, 1536), (9, 100)], ids=str)
def test_swiglu(dev, shape, dtype):
    M, K = shape
    g = torch.Generator().manual_seed(K)
    x = (3 * torch.randn(M, 2 * K, generator=g)).to(dtype)
    x[0, 0] = -100.0
    x[0, 1 % K] = 90.0
    q, s = run(x.to(dev), K, swiglu=True)
    v64 = torch.sigmoid(x.double()[:, :K]) * x.double()[:, :K] * x.double()[:, K:]
    rel = (x.double()[:, :K].abs() + 4) * 2.0 ** -23
    err = v64.abs() * rel + 1e-37
    rs = (blocks(v64).abs().amax(-1) / 448).clamp_min(2.0 ** -126)
    serr = blocks(err).amax(-1) / 448 + rs * 2.0 ** -23
    assert torch.all((s.double() - rs).abs() <= serr)
    sv = s.double().repeat_interleave(128, 1)[:, :K]
    back = q.view(F8).double() * sv
    tol = torch.maximum(v64.abs() * 2.0 ** -4, sv * 2.0 ** -10) * (1 + 2.0 ** -20) + err * (1 + 2.0 ** -4)
    worst = ((back - v64).abs() / tol).max().item()
    print(f"swiglu {shape} {dtype}: {worst:.3f} of the bound", flush=True)
    assert worst <= 1


def test_swiglu_nan_and_inf(dev):
    K = 256
    x = torch.ones(1, 2 * K)
    x[0, 3] = float("nan")
    x[0, K + 5] = float("inf")
    x[0, 7], x[0, K + 7] = -float("inf"), 2.0      # silu's limit is 0
    q, s = run(x.to(dev), K, swiglu=True)
    assert (q[0] == 0x7F).nonzero().flatten().tolist() == [3, 5]
    assert q[0, 7] in (0x00, 0x80)
    assert torch.isfinite(s).all()


def test_rows_beyond_32_bit_offsets(dev):
    """3 x 2^30 elements apart and a whole tensor of more than 2^32 bytes."""
    ld, K = 1 << 30, 256
    big = torch.empty(2 * ld + K, dtype=torch.bfloat16, device=dev)
    x = big.as_strided((3, K), (ld, 1))
    x.copy_(torch.randn(3, K, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(dev))
    same(run(x, K), reference(x.cpu().float()), "far rows")
    del big
    M, K = 140000, 16384 + 128
    x = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
    x.fill_(1.0)
    at = torch.tensor([0, 1, 65535, 65536, 130055, 130056, M - 1], device=dev)
    x[at] = torch.randn(7, K, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(dev)
    q = torch.zeros(M, K, dtype=torch.uint8, device=dev)
    s = torch.zeros(M, K // 128, device=dev)
    mg.moe_decode_quantize_fp8(x, q, s)
    torch.cuda.synchronize()
    same((q[at].cpu(), s[at].cpu()), reference(x[at].cpu().float()), "large")
    assert int((q == 0x7E).all(1).sum()) == M - 7      # 448


def test_capture_and_streams(dev):
    x = torch.randn(100, 512, device=dev, generator=torch.Generator(device=dev).manual_seed(5))
    q, s = torch.empty(100, 512, dtype=torch.uint8, device=dev), torch.empty(100, 4, device=dev)
    mg.moe_decode_quantize_fp8(x, q, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mg.moe_decode_quantize_fp8(x, q, s)
    for rep in range(3):
        x.mul_(-1.7)
        q.zero_()
        graph.replay()
        torch.cuda.synchronize()
        same((q.cpu(), s.cpu()), reference(x.cpu()), rep)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    mg.moe_decode_quantize_fp8(x, q2, s2, stream=st)
    st.synchronize()
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_refusals(dev):
    x, q, s = torch.zeros(4, 256, device=dev), torch.zeros(4, 256, dtype=torch.uint8, device=dev), torch.zeros(4, 2, device=dev)
    for bad in ((x.double(), q, s), (x, q.float(), s), (x, q, s.double()), (x, q, s[:, :1]), (x[:3], q, s), (x[:, :128], q, s),
                (torch.zeros(256, 4, device=dev).t(), q, s), (x, torch.zeros(4, 512, dtype=torch.uint8, device=dev)[:, ::2], s)):
        with pytest.raises(ValueError):
            mg.moe_decode_quantize_fp8(*bad)
    with pytest.raises(ValueError):
        mg.moe_decode_quantize_fp8(x, q, s, swiglu=True)   # x has to be twice as wide
    mg.moe_decode_quantize_fp8(x[:0], q[:0], s[:0])
