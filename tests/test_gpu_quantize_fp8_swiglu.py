"""GPU tests of moe_decode_quantize_fp8's SwiGLU.

v = SiLU(g) u with a = e^-|g|: the exponential 1 ulp and its correction's rounding
1/2, the constant in it |g| / 43, and at most 1/2 each for g a, 1 + a, the quotient
and the product with u: (3.5 + |g| / 43) 2^-23 relative.  In a block of one element the
scale is |v| / 448 rounded, 1/2 more: what it says of v is within (4 + |g| / 43) 2^-23.
"""
import pytest
import torch

import moe_gate_up_amd as mg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def test_error_at_every_size_of_gate(dev):
    """Blocks of one element, gates over the whole range whose exponential is a normal number."""
    M = 200000
    g = torch.Generator().manual_seed(1)
    x = torch.empty(M, 2)
    x[:, 0] = torch.cat([torch.linspace(-87, 87, M // 2), torch.randn(M // 2, generator=g) * 4])
    x[:, 1] = (1000 + 9000 * torch.rand(M, generator=g)) * torch.where(torch.rand(M, generator=g) < 0.5, 1.0, -1.0)
    q = torch.empty(M, 1, dtype=torch.uint8, device=dev)
    s = torch.empty(M, 1, device=dev)
    mg.moe_decode_quantize_fp8(x.to(dev), q, s, swiglu=True)
    gate, up = x.double().unbind(1)
    v = gate * torch.sigmoid(gate) * up
    off = (s[:, 0].cpu().double() * 448 / v.abs() - 1).abs() * 2.0 ** 23
    use = off / (4 + gate.abs() / 43)
    print(f"SwiGLU: off by {float(off.max()):.2f} 2^-23 at g = {float(gate[off.argmax()]):.2f}, {float(use.max()):.2f} of the bound", flush=True)
    assert float(use.max()) <= 1
    want = torch.where(v < 0, 0xFE, 0x7E).to(torch.uint8)      # 448, or -448
    assert torch.equal(q[:, 0].cpu(), want)


def power_of_two(s):
    """The smallest power of two that is not below s (float64; frexp: s = m 2^e, 1/2 <= m < 1)."""
    m, e = torch.frexp(s)
    return torch.where(m == 0.5, s, torch.ldexp(torch.ones_like(s), e))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 128), (5, 136), (65, 768), (9, 100), (33, 257)], ids=str)
def test_rows_apart_and_powers_of_two(dev, shape, dtype):
    """Rows with columns between them, a start that 16-byte loads cannot take, and power-of-two scales: the same codes and
    scales as of the packed rows, and those within their bounds.  A code's value is within half a step (2^-4 relative, or
    2^-10 scales among E4M3's subnormals) of v and v's own error."""
    M, K = shape
    g = torch.Generator().manual_seed(M + K)
    x = (3 * torch.randn(M, 2 * K, generator=g)).to(dtype)
    v = torch.sigmoid(x[:, :K].double()) * x[:, :K].double() * x[:, K:].double()
    err = v.abs() * (3.5 + x[:, :K].double().abs() / 43) * 2.0 ** -23 + 1e-36
    for pow2 in (False, True):
        first = None
        for pad, off in ((0, 0), (8, 0), (3, 0), (8, 1)):
            print(f"SwiGLU {shape} {dtype} pow2 {pow2} pads {pad} {off}", flush=True)
            wide = torch.full((M, 2 * K + pad + off), float("nan"), dtype=dtype, device=dev)
            wide[:, off:off + 2 * K] = x.to(dev)
            q = torch.full((M, K), 0xAA, dtype=torch.uint8, device=dev)
            s = torch.full((M, -(-K // 128)), -1.0, device=dev)
            mg.moe_decode_quantize_fp8(wide[:, off:off + 2 * K], q, s, swiglu=True, pow2=pow2)
            first = first or (q, s)
            assert torch.equal(q, first[0]) and torch.equal(s, first[1])
        q, s = first[0].cpu(), first[1].cpu().double()
        blocks = lambda t: torch.nn.functional.pad(t, (0, -K % 128)).view(M, -1, 128).amax(-1)   # noqa: E731
        low, high = blocks((v.abs() - err).clamp_min(0)) / 448 * (1 - 2.0 ** -24), blocks(v.abs() + err) / 448 * (1 + 2.0 ** -24)
        if pow2:
            low, high = power_of_two(low), power_of_two(high)
        assert bool(((low <= s) & (s <= high)).all())
        each = s.repeat_interleave(128, 1)[:, :K]
        back = q.view(torch.float8_e4m3fn).double() * each
        tol = torch.maximum(v.abs() * 2.0 ** -4, each * 2.0 ** -10) * (1 + 2.0 ** -20) + err * (1 + 2.0 ** -4)
        assert bool(((back - v).abs() <= tol).all())
