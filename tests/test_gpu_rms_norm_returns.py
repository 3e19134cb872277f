"""GPU tests of what moe_decode_rms_norm returns, and of its weight's gradient over long chains of rows.

dweight's tolerance above 4096 columns, where a workgroup holds one row at a time (R = 1): each of 256 workgroups adds up M / 256
rows in FP32 (FP64 behind), each term within 2 u, u = 2^-24: M / 256 + 2 u of the terms' magnitudes; R rows at a time up to there,
R = 16, 8, 4, 2 up to 512, 1024, 2048, 4096 columns: M / (256 R) additions and log2 R more.
"""
import pytest
import torch

import moe_gate_up_amd as mg
from tests.test_gpu_rms_norm import EPS, TINY, U, dev, make  # noqa: F401

pytestmark = pytest.mark.gpu


def test_outputs_as_given(dev):  # noqa: F811
    x, res, w = make(1, 6, 256, torch.bfloat16, torch.bfloat16, dev)
    y, total, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(6, device=dev)
    q, s = torch.empty(6, 256, dtype=torch.uint8, device=dev), torch.empty(6, 2, device=dev)
    got = mg.moe_decode_rms_norm(x, w, EPS, y=y, q=q, scales=s, residual=res, sum_out=total, rstd=rstd)
    assert all(a is b for a, b in zip(got, (y, q, s, total, rstd))) and len(got) == 5
    got = mg.moe_decode_rms_norm(x, w, EPS, q=q, scales=s)
    assert got[1] is q and got[2] is s and got[0] is got[3] is got[4] is None


@pytest.mark.parametrize("shape", [(40000, 4104), (20000, 8200), (70000, 1000)], ids=str)
def test_weight_gradient_of_many_rows(dev, shape):  # noqa: F811
    M, H = shape
    g = torch.Generator(device=dev).manual_seed(M)
    r, dy = (torch.randn(M, H, generator=g, device=dev).to(torch.bfloat16) + 0.5 for _ in range(2))   # terms mostly of one sign
    w = torch.ones(H, dtype=torch.bfloat16, device=dev)
    rstd = 1 + torch.rand(M, generator=g, device=dev)
    dx, dw = torch.empty_like(r), torch.empty(H, device=dev)
    mg.moe_decode_rms_norm_backward(dy, r, w, rstd, dx, dw)
    ref, size = (torch.zeros(H, dtype=torch.float64, device=dev) for _ in range(2))
    for i in range(0, M, 2000):
        t = dy[i:i + 2000].double() * (r[i:i + 2000].double() * rstd[i:i + 2000, None].double())
        ref += t.sum(0)
        size += t.abs().sum(0)
    R = 16 if H <= 512 else 8 if H <= 1024 else 4 if H <= 2048 else 2 if H <= 4096 else 1
    chain = -(-M // (256 * R)) + R.bit_length() - 1 + 2
    assert bool(((dw.double() - ref).abs() <= chain * U * size + TINY).all())
