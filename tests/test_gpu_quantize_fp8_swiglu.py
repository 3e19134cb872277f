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
