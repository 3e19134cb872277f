"""GPU tests of moe_decode_route_experts and its gradient with sigmoid scores far below FP32's smallest normal number: renormalised
weights are the scores' quotients all the same.  Against float64, with the tolerances of test_gpu_route_experts.py.

Without renorm a score s below 2^-126 counts as 0 and the result is scale * s: a weight is off by up to scale * 2^-126 = 2.5 *
1.2e-38 on top of its relative error, a gradient scale * g * s (1 - s) by |g| times as much.
"""
import pytest
import torch

import moe_gate_up_amd as mg
from tests.test_gpu_route_experts import INF, REL, TINY, check, dev, gradient, make, reference, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(64, 6, 1, 1), (128, 8, 8, 4), (512, 8, 1, 1), (96, 40, 2, 1)], ids=str)
def test_quotients_of_small_scores(dev, shape, dtype):  # noqa: F811
    """Rows whose logits lie around 0 to -600, where float64 has the scores; some experts ruled out."""
    E, k, groups, top = shape
    T = 200
    l = (make(E, T, E, torch.float32, torch.device("cpu")) - torch.linspace(0, 600, T)[:, None]).to(dtype)
    l[::7, 1::3] = -INF
    bias = (0.1 * torch.randn(E, generator=torch.Generator().manual_seed(E))).to(dev)
    for b in (None, bias):
        print(f"small {shape} {dtype} bias={b is not None}", flush=True)
        check(l.to(dev), b, k, True, True, groups, top, True, 2.5)
        grad = torch.randn(T, k, generator=torch.Generator().manual_seed(k)).to(dev)
        ids, w, d = run(l.to(dev), b, k, True, False, groups, top, True, 2.5, grad)
        rid, rw = reference(l, b, k, True, False, groups, top, True, 2.5)
        assert torch.equal(ids.cpu().long(), rid)
        assert bool(((w.cpu().double() - rw).abs() <= REL * rw + 2.5 * TINY).all())
        rd, size = gradient(l, rid, grad, True, False, 2.5)
        eps = torch.finfo(dtype).eps / 2 if dtype == torch.bfloat16 else 0
        off = 3 * REL * size + 2.5 * float(grad.abs().max()) * TINY
        assert bool(((d.cpu().double() - rd).abs() <= off + eps * (rd.abs() + off)).all())


def test_no_score_left(dev):  # noqa: F811
    """Where 64 bits have no score either the weights and the gradient are 0."""
    for low in (-800.0, -1e5, torch.finfo(torch.float32).min, -INF):
        l = torch.full((5, 48), low, device=dev)
        l[1] += torch.arange(48, device=dev)
        l[2, 20:] = -INF
        check(l, None, 6, True, True)
        check(l, torch.linspace(-1, 1, 48).to(dev), 6, True, True, 4, 2, True)


def test_gradient_of_ids_from_elsewhere(dev):  # noqa: F811
    """Repeated ids and ids out of range among small scores: d w_j / d l_e for the ids as they stand."""
    l = make(1, 3, 20, torch.float32, dev) - 120
    ids = torch.tensor([[3, 3, 5], [-1, 20, 2], [7, -5, 7]], dtype=torch.int32, device=dev)
    grad = torch.randn(3, 3, generator=torch.Generator().manual_seed(6)).to(dev)
    d = torch.full_like(l, 4.0)
    mg.moe_decode_route_experts_backward(l, ids, grad, d, sigmoid=True)
    for t in range(3):
        on = [j for j in range(3) if 0 <= int(ids[t, j]) < 20]
        at, g = ids[t, on].cpu().long(), grad[t, on].cpu().double()
        w = torch.softmax(l[t].cpu().double()[at], 0)   # so far down a sigmoid is e^l
        term = w * (g - (g * w).sum())
        ref = torch.zeros(20, dtype=torch.float64).index_add_(0, at, term)
        assert bool(((d[t].cpu().double() - ref).abs() <= 3 * 110 * 2.0 ** -24 * (g.abs().sum()) + 1.2e-38).all()), t
